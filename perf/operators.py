"""Workloads of the serving operators: low-rank adapters beside a projection, appending to an
8-bit paged key/value cache, and attention over that cache.

Each case is run either in a plain form (elementary torch operations in fp32) or, where ``own``
is true, through the library's entry points.  ``exact`` gives the same outputs from the
definitions in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda:0"
CODE_MAX = {"fp8": 448.0, "int8": 127.0}
CODE_TYPE = {"fp8": torch.float8_e4m3fn, "int8": torch.int8}


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # adapters: a few requests decoding, each with its own adapter; latency counts
        {"name": "adapter_decode_4", "op": "adapter", "tokens": 4, "spans": 4, "n": 4, "rank": 16,
         "d_in": 4096, "d_out": 4096, "out": "f16", "mix": 1},
        # adapters: a decode batch over the down projection of the MLP, ranks mixed, some
        # requests without an adapter
        {"name": "adapter_decode_mlp", "op": "adapter", "tokens": 61, "spans": 61, "n": 24,
         "rank": 64, "d_in": 11008, "d_out": 4096, "out": "f32", "mix": 2},
        # adapters: prompts of several requests in one batch, lengths odd
        {"name": "adapter_prefill", "op": "adapter", "tokens": 4099, "spans": 7, "n": 8,
         "rank": 32, "d_in": 4096, "d_out": 4096, "out": "f16", "mix": 3},
        # cache append: one token for each request of a decode batch
        {"name": "append_decode_32", "op": "append", "kind": "fp8", "req": 32, "new": 1,
         "cached": 700, "heads": 32, "dim": 128, "page": 64, "src": "f16", "mix": 4},
        # cache append: a few odd tokens for each request, small pages, fp32 projections
        {"name": "append_chunks_int8", "op": "append", "kind": "int8", "req": 12, "new": 37,
         "cached": 250, "heads": 8, "dim": 128, "page": 16, "src": "f32", "mix": 5},
        # cache append: whole prompts
        {"name": "append_prefill", "op": "append", "kind": "fp8", "req": 6, "new": 1400,
         "cached": 0, "heads": 32, "dim": 128, "page": 64, "src": "f16", "mix": 6},
        # attention: one request decoding over a short cache; latency counts
        {"name": "attend_decode_1", "op": "attend", "kind": "fp8", "req": 1, "new": 1,
         "cached": 776, "heads": 32, "group": 1, "dim": 128, "page": 64, "window": 0, "sinks": 0,
         "out": "f16", "mix": 0},
        # attention: a decode batch, lengths from hundreds to 8192
        {"name": "attend_decode_32", "op": "attend", "kind": "fp8", "req": 32, "new": 1,
         "cached": 8191, "heads": 32, "group": 1, "dim": 128, "page": 64, "window": 0, "sinks": 0,
         "out": "f16", "mix": 8},
        # attention: streaming decode, five query heads for each cached head, a window and four
        # first tokens, pages between them given back
        {"name": "attend_window_int8", "op": "attend", "kind": "int8", "req": 24, "new": 1,
         "cached": 30001, "heads": 8, "group": 5, "dim": 128, "page": 16, "window": 4096,
         "sinks": 4, "out": "f16", "mix": 9},
        # attention: one very long request, a few drafted tokens verified at once
        {"name": "attend_long_draft", "op": "attend", "kind": "fp8", "req": 1, "new": 4,
         "cached": 131067, "heads": 8, "group": 4, "dim": 128, "page": 128, "window": 0,
         "sinks": 0, "out": "f16", "mix": 0},
        # attention: chunks of prompts of several requests, some of it cached before
        {"name": "attend_prefill", "op": "attend", "kind": "fp8", "req": 3, "new": 2048,
         "cached": 1021, "heads": 8, "group": 4, "dim": 128, "page": 64, "window": 0, "sinks": 0,
         "out": "f16", "mix": 11},
        # attention: a prompt under a window with sinks, small heads, fp32 output
        {"name": "attend_prefill_window", "op": "attend", "kind": "int8", "req": 2, "new": 3001,
         "cached": 0, "heads": 16, "group": 1, "dim": 64, "page": 32, "window": 512, "sinks": 4,
         "out": "f32", "mix": 12},
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    mix = rng.randrange(1, 1 << 20)
    op = rng.choice(["adapter", "append", "attend", "attend"])
    if op == "adapter":
        tokens = _log_int(rng, 1, 4099)
        spans = tokens if tokens <= 64 else rng.randint(1, 12)
        return {"op": op, "tokens": tokens, "spans": spans, "n": _log_int(rng, 1, 24),
                "rank": rng.choice([8, 16, 32, 64]), "d_in": 8 * _log_int(rng, 32, 1376),
                "d_out": _log_int(rng, 250, 4100), "out": rng.choice(["f16", "f32"]), "mix": mix}
    kind, page = rng.choice(["fp8", "int8"]), rng.choice([16, 32, 64, 128])
    dim, heads = rng.choice([64, 96, 128]), rng.choice([1, 2, 3, 8, 16, 32])
    if op == "append":
        total = _log_int(rng, 1, 8192)
        req = min(total, _log_int(rng, 1, 64))
        return {"op": op, "kind": kind, "req": req, "new": max(1, total // req),
                "cached": rng.choice([0, _log_int(rng, 1, 900)]), "heads": heads, "dim": dim,
                "page": page, "src": rng.choice(["f16", "f32"]), "mix": mix}
    group = rng.choice([1, 1, 4, 5, 8])
    window = rng.choice([0, 0, _log_int(rng, 100, 4096)])
    case = {"op": op, "kind": kind, "heads": min(heads, 32 // group), "group": group, "dim": dim,
            "page": page, "window": window, "sinks": rng.choice([0, 4, 7]) if window else 0,
            "out": rng.choice(["f16", "f32"]), "mix": mix}
    if rng.random() < 0.5:  # decode, or a few drafted tokens
        req = _log_int(rng, 1, 32)
        case |= {"req": req, "new": rng.choice([1, 1, 1, 3]),
                 "cached": _log_int(rng, 30, 120000 // req)}
    else:
        req = rng.randint(1, 4)
        case |= {"req": req, "new": _log_int(rng, 20, 2600 // req),
                 "cached": rng.choice([0, _log_int(rng, 30, 2048)])}
    return case


# ------------------------------------------------------------------------------------ inputs

def _spread(rng, total, parts):
    """`total` in `parts` whole numbers of one or more, uneven."""
    cuts = sorted(rng.sample(range(1, total), parts - 1)) if parts > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _adapter_plan(case):
    """Adapter of each token, and the ranks: the tokens of a request stand together."""
    rng = random.Random(case["mix"])
    n, r = case["n"], case["rank"]
    ranks = [max(1, (r, r // 2, r, r // 4, r - 3)[i % 5]) if case["mix"] != 1 else r
             for i in range(n)]
    ids = []
    for length in _spread(rng, case["tokens"], case["spans"]):
        a = rng.randrange(n) if case["spans"] != n else len(set(ids))
        ids += [-1 if case["mix"] % 2 == 0 and rng.random() < 0.1 else a] * length
    return ids, ranks


def _lengths(case):
    """(cached, new) tokens of each request: the first has the most, the others fewer."""
    rng = random.Random(case["mix"])
    cached, new = [], []
    for i in range(case["req"]):
        f = 1.0 if i == 0 else rng.uniform(0.06, 1.0)
        cached.append(int(case["cached"] * f))
        new.append(case["new"] if case["new"] < 8 else max(1, int(case["new"] * (
            1.0 if i == 0 else rng.uniform(0.5, 1.0)))))
    return cached, new


def _encode(x, scale, kind):
    """Nearest code of x / scale (0 where the scale is 0), as a value of the code's type."""
    q = torch.where(scale > 0, x / torch.where(scale > 0, scale, torch.ones_like(scale)),
                    torch.zeros_like(x))
    if kind == "fp8":
        return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.round().clamp(-127.0, 127.0).to(torch.int8)


def _cache(case, cached, total, gen):
    """A pool of pages holding every request's first tokens: codes, scales, page table."""
    req, page, heads, dim, kind = (case[k] for k in ("req", "page", "heads", "dim", "kind"))
    need = [-(-t // page) for t in total]
    pool = sum(need) + max(2, sum(need) // 16)
    order = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((req, max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    chan = torch.exp(0.4 * torch.randn(heads, 1, dim, generator=gen, device=DEV))
    mean = torch.randn(heads, 1, dim, generator=gen, device=DEV)
    codes = {"k": torch.empty(pool, heads, page, dim, dtype=CODE_TYPE[kind], device=DEV),
             "v": torch.empty(pool, heads, dim, page, dtype=CODE_TYPE[kind], device=DEV)}
    scales = {n: torch.empty(pool, heads, dtype=torch.float32, device=DEV) for n in ("k", "v")}
    first = torch.zeros(pool, dtype=torch.bool, device=DEV)
    first[table[:, 0].long()] = True
    step = max(1, (1 << 27) // (heads * page * dim))
    for p in range(0, pool, step):
        for n in ("k", "v"):
            x = torch.randn(min(step, pool - p), heads, page, dim, generator=gen, device=DEV)
            if n == "k":  # uneven channels, and first tokens that many queries look at
                x = x * chan
                x[:, :, :4] += 1.5 * mean * first[p:p + step, None, None, None]
            s = x.abs().amax((2, 3)) / CODE_MAX[kind]
            scales[n][p:p + step] = s
            y = _encode(x, s[:, :, None, None], kind)
            if n == "v":
                y = y.view(torch.uint8).transpose(2, 3).contiguous().view(CODE_TYPE[kind])
            codes[n].view(torch.uint8)[p:p + step] = y.view(torch.uint8)
    return codes, scales, table, mean


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(new):
    return [0] + [int(x) for x in np.cumsum(new)]


def _inputs(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed * 1000003 + case["mix"])
    rand = lambda *shape: torch.randn(*shape, generator=gen, device=DEV)  # noqa: E731
    if case["op"] == "adapter":
        ids, ranks = _adapter_plan(case)
        n, r, d_in, d_out, T = (case[k] for k in ("n", "rank", "d_in", "d_out", "tokens"))
        out = torch.float16 if case["out"] == "f16" else torch.float32
        r8 = -(-r // 8) * 8
        return {"X": (rand(T, d_in) * torch.exp(0.3 * rand(1, d_in))).half(),
                "A": (rand(n, r8, d_in) / math.sqrt(d_in)).half(),
                "B": (0.1 * rand(n, d_out, r8)).half(), "base": rand(T, d_out).to(out),
                "rank": _ints(ranks), "scale": 16.0 / _ints(ranks).float(), "ids": _ints(ids)}
    cached, new = _lengths(case)
    total = [a + b for a, b in zip(cached, new)]
    codes, scales, table, mean = _cache(case, cached, total, gen)
    n_tok, heads, dim = sum(new), case["heads"], case["dim"]
    s = {"codes": codes, "scales": scales, "table": table, "start": _ints(_starts(new)),
         "cached": _ints(cached), "length": _ints(total), "host": (cached, new)}
    if case["op"] == "append":
        src = torch.float16 if case["src"] == "f16" else torch.float32
        s["K"] = (rand(n_tok, heads, dim) * 1.1).to(src).reshape(n_tok, heads * dim)
        s["V"] = rand(n_tok, heads, dim).to(src).reshape(n_tok, heads * dim)
    else:
        q = rand(n_tok, heads, case["group"], dim) + 0.5 * mean.transpose(0, 1)[:, :, None].reshape(
            1, heads, 1, dim)
        s["Q"] = q.half().reshape(n_tok, heads * case["group"] * dim)
        if case["window"]:  # pages that no query sees any more have been given back
            page, keep = case["page"], -(-case["sinks"] // case["page"])
            for i in range(case["req"]):
                dead = max(0, cached[i] + 1 - case["window"]) // page
                if dead > keep:
                    s["table"][i, keep:dead] = -1
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:  # the library's view of the same tensors, and the workspace that a program keeps
        from dictionary_factored_sparse_amd import binding as B
        if case["op"] == "adapter":
            s["own"] = B.DeviceAdapters(s["A"], s["B"], s["rank"], s["scale"])
            s["ws"] = B.adapter_workspace(case["tokens"], s["own"], DEV)
        else:
            s["own"] = B.DeviceKV8(s["codes"]["k"].view(torch.uint8),
                                   s["codes"]["v"].view(torch.uint8), s["scales"]["k"],
                                   s["scales"]["v"], case["kind"])
        if case["op"] == "attend":
            s["ws"] = B.kv8_attention_workspace(s["own"], case["req"], s["Q"].shape[0],
                                                case["heads"] * case["group"], DEV)
    return s


# ------------------------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    return {"adapter": _adapter, "append": _append, "attend": _attend}[case["op"]](s, case)


def _adapter(s, case):
    out = torch.float16 if case["out"] == "f16" else torch.float32
    if own:
        from dictionary_factored_sparse_amd import binding as B
        return B.dict_adapter_forward(s["X"], s["own"], s["ids"], base=s["base"], ydtype=out,
                                      ws=s["ws"])
    n, r, d_in = s["A"].shape
    d_out = s["B"].shape[1]
    mine = s["ids"][:, None] == torch.arange(n, device=DEV)
    used = torch.arange(r, device=DEV) < s["rank"][:, None]
    weight = (mine[:, :, None] & used) * s["scale"][:, None]
    u = s["X"].float() @ s["A"].float().reshape(n * r, d_in).T
    u = u * weight.reshape(-1, n * r)
    y = s["base"].float() + u @ s["B"].float().transpose(1, 2).reshape(n * r, d_out)
    return y.to(out)


def _append(s, case):
    if own:
        from dictionary_factored_sparse_amd import binding as B
        B.kv8_append(s["own"], s["K"], s["V"], s["start"], s["cached"], s["table"])
        return [s["codes"]["k"], s["scales"]["k"], s["codes"]["v"], s["scales"]["v"]]
    page, heads, dim, kind = (case[k] for k in ("page", "heads", "dim", "kind"))
    host_cached, host_new = s["host"]
    touched = sum((c + n - 1) // page - c // page + 1 for c, n in zip(host_cached, host_new) if n)
    start, cached = s["start"].long(), s["cached"].long()
    new = start[1:] - start[:-1]
    count = torch.where(new > 0, (cached + new - 1) // page - cached // page + 1, 0)
    req = torch.repeat_interleave(torch.arange(len(new), device=DEV), count, output_size=touched)
    logical = (cached // page)[req] + torch.arange(touched, device=DEV) - (
        torch.cumsum(count, 0) - count)[req]
    where = s["table"].long()[req, logical]
    pos = logical[:, None] * page + torch.arange(page, device=DEV)
    is_old = pos < cached[req][:, None]
    is_new = (pos < (cached + new)[req][:, None]) & ~is_old
    row = (start[:-1][req][:, None] + pos - cached[req][:, None]).clamp(0, s["K"].shape[0] - 1)
    for n, src in (("k", s["K"]), ("v", s["V"])):
        # (touched, heads, page, dim) for keys; values are held with the page's tokens last
        x = src.float().reshape(-1, heads, dim)[row].permute(0, 2, 1, 3)
        fresh, held = is_new[:, None, :, None], is_old[:, None, :, None]
        if n == "v":
            x, fresh, held = (t.transpose(2, 3) for t in (x, fresh, held))
        x = torch.where(fresh, x, 0.0)
        need = x.abs().amax((2, 3)) / CODE_MAX[kind]
        before = s["scales"][n][where] * is_old.any(1)[:, None]
        scale = torch.maximum(need, before)
        codes = s["codes"][n].view(torch.uint8)[where]
        wide = scale[:, :, None, None]
        again = _encode(codes.view(CODE_TYPE[kind]).float() * before[:, :, None, None], wide, kind)
        grown = held & (need > before)[:, :, None, None]
        codes = torch.where(grown, again.view(torch.uint8), codes)
        codes = torch.where(fresh, _encode(x, wide, kind).view(torch.uint8), codes)
        s["codes"][n].view(torch.uint8)[where] = codes
        s["scales"][n][where] = scale
    return [s["codes"]["k"], s["scales"]["k"], s["codes"]["v"], s["scales"]["v"]]


def _attend(s, case):
    heads, group, dim, page = (case[k] for k in ("heads", "group", "dim", "page"))
    out = torch.float16 if case["out"] == "f16" else torch.float32
    if own:
        from dictionary_factored_sparse_amd import binding as B
        return B.kv8_attention(s["own"], s["Q"], s["start"], s["length"], s["table"],
                               heads * group, window=case["window"], sinks=case["sinks"],
                               odtype=out, ws=s["ws"])
    cached, new = s["host"]
    req, most, length = len(new), max(new), s["table"].shape[1] * page
    where = s["table"].long().clamp(min=0)
    k = s["codes"]["k"][where].float() * s["scales"]["k"][where][..., None, None]
    k = k.permute(0, 2, 1, 3, 4).reshape(req, heads, length, dim)
    v = s["codes"]["v"][where].float() * s["scales"]["v"][where][..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(req, heads, length, dim)
    start, n_new = s["start"][:-1].long(), (s["start"][1:] - s["start"][:-1]).long()
    at = torch.arange(most, device=DEV)
    row = (start[:, None] + at).clamp(max=s["Q"].shape[0] - 1)
    q = s["Q"].float().reshape(-1, heads, group, dim)[row]              # (req, most, heads, ..)
    q = q.permute(0, 2, 3, 1, 4).reshape(req, heads, group * most, dim)
    pos = (s["length"].long() - n_new)[:, None] + at                    # (req, most)
    key = torch.arange(length, device=DEV)
    seen = key <= pos[:, :, None]
    if case["window"]:
        seen = seen & ((pos[:, :, None] - key < case["window"]) | (key < case["sinks"]))
    seen = seen[:, None].expand(req, group, most, length).reshape(req, 1, group * most, length)
    score = torch.where(seen, q @ k.transpose(2, 3).contiguous() / math.sqrt(dim), -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    o = (e @ v) / e.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.reshape(req, heads, group, most, dim).permute(0, 3, 1, 2, 4)  # (req, most, heads, ..)
    o = o[at < n_new[:, None]] if min(new) < most else o.reshape(req * most, heads, group, dim)
    return o.reshape(-1, heads * group * dim).to(out)


# ------------------------------------------------------------------------------------ accounting

def _visible(case, cached, new):
    """(keys that some query of the request sees, sum over its queries of the keys seen)."""
    pos = cached + np.arange(new, dtype=np.int64)
    if not case["window"]:
        return cached + new, int((pos + 1).sum())
    low = np.maximum(0, pos - case["window"] + 1)
    sinks = np.minimum(case["sinks"], low)
    return cached + new - int(low[0]) + int(min(case["sinks"], low[0])), int(
        (pos + 1 - low + sinks).sum())


def work(case):
    if case["op"] == "adapter":
        ids, ranks = _adapter_plan(case)
        both = case["d_in"] + case["d_out"]
        live = [a for a in ids if a >= 0]
        size = 2 if case["out"] == "f16" else 4
        return {"bytes": 2 * both * sum(ranks[a] for a in set(live)) + 2 * case["d_in"] * len(live)
                + 2 * size * case["tokens"] * case["d_out"] + 4 * case["tokens"],
                "flops": 2 * both * sum(ranks[a] for a in live)}
    cached, new = _lengths(case)
    heads, dim, page = case["heads"], case["dim"], case["page"]
    if case["op"] == "append":
        size = 2 if case["src"] == "f16" else 4
        pages = sum((c + n - 1) // page - c // page + 1 for c, n in zip(cached, new))
        return {"bytes": 2 * heads * (sum(new) * dim * (size + 1) + 8 * pages),
                "flops": 4 * heads * dim * sum(new)}
    seen = [_visible(case, c, n) for c, n in zip(cached, new)]
    size = 2 + (2 if case["out"] == "f16" else 4)
    keys, pairs = sum(k for k, _ in seen), sum(p for _, p in seen)
    return {"bytes": 2 * heads * keys * dim + 8 * heads * (keys // page)
            + size * sum(new) * heads * case["group"] * dim,
            "flops": 4 * dim * heads * case["group"] * pairs}


# ------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "adapter":
        y = s["base"].double()
        ids, ranks = _adapter_plan(case)
        ids = np.array(ids)
        for a in sorted(set(ids[ids >= 0].tolist())):
            rows = torch.from_numpy(np.flatnonzero(ids == a)).to(DEV)
            u = s["X"][rows].double() @ s["A"][a, :ranks[a]].double().T
            y[rows] += float(s["scale"][a]) * (u @ s["B"][a, :, :ranks[a]].double().T)
        return y
    cached, new = s["host"]
    page, heads, dim, kind = (case[k] for k in ("page", "heads", "dim", "kind"))
    table = s["table"].cpu().numpy()
    if case["op"] == "append":
        out = []
        for n, src in (("k", s["K"]), ("v", s["V"])):
            held, scales = s["codes"][n].double(), s["scales"][n].double()
            if n == "v":
                held = held.transpose(2, 3).contiguous()
            row = 0
            for i in range(len(new)):
                p = cached[i]
                while p < cached[i] + new[i]:
                    at, lo = int(table[i, p // page]), p % page
                    m = min(page - lo, cached[i] + new[i] - p)
                    x = src[row:row + m].double().reshape(m, heads, dim).transpose(0, 1)
                    was = scales[at] if lo else torch.zeros_like(scales[at])
                    now = torch.maximum(was, x.abs().amax((1, 2)) / CODE_MAX[kind])
                    if kind == "fp8":
                        # a code that is kept stays; one that is written again is the nearest
                        # value of its type
                        safe = torch.where(now > 0, now, 1.0)[:, None, None]
                        older = held[at, :, :lo]
                        again = _nearest8(older * was[:, None, None] / safe)
                        held[at, :, :lo] = torch.where((now > was)[:, None, None], again, older)
                        held[at, :, lo:lo + m] = _nearest8(x / safe)
                    scales[at] = now
                    p, row = p + m, row + m
            codes = None if kind == "int8" else (held.transpose(2, 3) if n == "v" else held)
            out += [codes, scales]
        return out
    o = torch.zeros(sum(new), heads * case["group"], dim, dtype=torch.float64, device=DEV)
    row = 0
    for i in range(len(new)):
        total = cached[i] + new[i]
        key = np.arange(total)
        seen = key[None, :] <= (cached[i] + np.arange(new[i]))[:, None]
        if case["window"]:
            far = (cached[i] + np.arange(new[i]))[:, None] - key[None, :] >= case["window"]
            seen &= ~far | (key < case["sinks"])[None, :]
        seen = torch.from_numpy(seen).to(DEV)
        pages = torch.from_numpy(np.maximum(table[i, key // page], 0).astype(np.int64)).to(DEV)
        slot = torch.from_numpy(key % page).to(DEV)
        q = s["Q"][row:row + new[i]].double().reshape(new[i], heads, case["group"], dim)
        for h in range(heads):
            k, v = (s["codes"][n].view(torch.uint8)[where].view(CODE_TYPE[kind]).double()
                    * s["scales"][n][pages, h, None].double()
                    for n, where in (("k", (pages, h, slot)),
                                     ("v", (pages, h, slice(None), slot))))
            for g in range(case["group"]):
                p = torch.softmax(torch.where(seen, q[:, h, g] @ k.T / math.sqrt(dim),
                                              -math.inf), 1)
                o[row:row + new[i], h * case["group"] + g] = p @ v
        row += new[i]
    return o.reshape(sum(new), -1)


def _nearest8(x):
    """The E4M3 value nearest to each x, ties to even, at most 448 in size, in 64 bits."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=448.0)
