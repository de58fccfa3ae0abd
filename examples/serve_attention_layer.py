"""One attention layer of a compressed model, served: q, k and v projections from three shared
dictionaries (dict_multi_forward), low-rank adapters of the requests beside them
(dict_adapter_forward), rotary positions, the 8-bit paged cache (kv8_append), attention with a
sliding window and first tokens that stay visible (kv8_attention), and the output projection
(dict_proj_forward).

    python examples/serve_attention_layer.py

Three requests send prompts of different lengths in one batch, then decode token by token; pages
are handed out as the requests grow and taken back once the window has left them.  Every step is
compared with the same layer in float64 over the decoded cache.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dictionary_factored_sparse_amd import binding as B  # noqa: E402

D_MODEL, HEADS, HEAD_DIM, ATOMS, PAGE = 512, 8, 64, 256, 16


class Pages:
    """Free pages of the cache and each request's row of the page table."""

    def __init__(self, n_pages, n_req, per_req, device):
        self.free = list(range(n_pages))
        self.table = torch.full((n_req, per_req), -1, dtype=torch.int32)
        self.device = device

    def grow(self, req, length):
        """Pages for the request's first `length` tokens (those given back stay away)."""
        for i in range((length + PAGE - 1) // PAGE):
            if self.table[req, i] == -1:
                self.table[req, i] = self.free.pop()

    def shrink(self, req, length, window, sinks):
        """Take back the pages that no later token sees."""
        for i in range(-(-sinks // PAGE), max(0, length - window + 1) // PAGE):
            if self.table[req, i] >= 0:
                self.free.append(int(self.table[req, i]))
                self.table[req, i] = -2       # no page, and none wanted

    def device_table(self):
        return self.table.to(self.device)


class Layer:
    """Weights of the layer (random), in the library's formats."""

    def __init__(self, device, seed=0, n_adapters=2, rank=8):
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.dense = {}
        self.dicts, self.coefs = [], []
        for name in ("q", "k", "v", "o"):
            atoms = (rand(ATOMS, D_MODEL) / D_MODEL ** 0.5).half()
            coef = (rand(ATOMS, D_MODEL) * (torch.rand(ATOMS, D_MODEL, generator=g) < 0.3)
                    / (0.3 * ATOMS) ** 0.5).half()
            self.dicts.append(B.DeviceDict.from_atoms(atoms.to(device)))
            self.coefs.append(B.dict_pack_csc(coef.to(device)))
            self.dense[name] = (atoms.double().T @ coef.double()).to(device)
        self.adapters = {}
        for name in ("q", "v"):
            A = (rand(n_adapters, rank, D_MODEL) / D_MODEL ** 0.5).half().to(device)
            Bm = (0.2 * rand(n_adapters, D_MODEL, rank)).half().to(device)
            self.adapters[name] = B.DeviceAdapters(
                A, Bm, torch.tensor([rank, rank // 2], dtype=torch.int32, device=device),
                torch.full((n_adapters,), 2.0, device=device))


def rotate(x, pos):
    """Rotary positions on (tokens, heads * head_dim), in the tensor's type."""
    half = HEAD_DIM // 2
    freq = 10000.0 ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    angle = pos.double()[:, None, None] * freq
    y = x.double().reshape(len(x), HEADS, 2, half)
    a, b = y[:, :, 0], y[:, :, 1]
    out = torch.stack([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], 2)
    return out.reshape(len(x), HEADS * HEAD_DIM).to(x.dtype)


def step(layer, kv, X, ids, start, cached, table, window, sinks):
    """One call of the layer: X (tokens, d_model) f16, the rows of request r are start[r] ..
    start[r + 1] - 1, and cached[r] tokens of it are in the cache.  Returns (q, output)."""
    q, k, v = B.dict_multi_forward([X], layer.dicts[:3], layer.coefs[:3])
    for name, y in (("q", q), ("v", v)):      # beside the shared projection, in place
        B.dict_adapter_forward(X, layer.adapters[name], ids, base=y, Y=y)
    new = start[1:] - start[:-1]
    row = torch.arange(len(X), device=X.device)
    req = torch.searchsorted(start[1:].contiguous(), row, right=True)
    pos = cached[req] + row - start[req]
    q, k = rotate(q, pos), rotate(k, pos)
    B.kv8_append(kv, k, v, start, cached, table)
    o = B.kv8_attention(kv, q, start, cached + new, table, HEADS, window=window, sinks=sinks)
    return q, B.dict_proj_forward(o, layer.dicts[3], layer.coefs[3])


def decoded(kv, table, length):
    """(keys, values) of one request's first tokens in float64, (length, heads, head_dim); tokens
    whose page is gone are zero."""
    j = torch.arange(length, device=table.device)
    pg = table[j // PAGE].long()
    here, pg = pg >= 0, pg.clamp(min=0)
    kind = torch.float8_e4m3fn if kv.kind == "fp8" else torch.int8
    k = kv.k.view(kind)[pg, :, j % PAGE].double() * kv.kscale[pg].double()[:, :, None]
    v = kv.v.view(kind)[pg, :, :, j % PAGE].double() * kv.vscale[pg].double()[:, :, None]
    return k * here[:, None, None], v * here[:, None, None]


def check(layer, kv, q, y, start, length, table, window, sinks):
    """Largest error of the step's output over its largest value, against float64."""
    want = []
    for r in range(len(length)):
        n, total = int(start[r + 1] - start[r]), int(length[r])
        k, v = decoded(kv, table[r], total)
        rows = q[int(start[r]):int(start[r + 1])].double().reshape(n, HEADS, HEAD_DIM)
        pos = torch.arange(total - n, total, device=q.device)[:, None]
        j = torch.arange(total, device=q.device)[None]
        seen = (j <= pos) & ((pos - j < window) | (j < sinks))
        s = torch.einsum("nhd,jhd->hnj", rows, k) / HEAD_DIM ** 0.5
        p = torch.softmax(torch.where(seen, s, -torch.inf), -1)
        want.append(torch.einsum("hnj,jhd->nhd", p, v).reshape(n, -1) @ layer.dense["o"])
    want = torch.cat(want)
    return float((y.double() - want).abs().max() / want.abs().max())


def main(kind="fp8", steps=40, window=48, sinks=4, device="cuda:0", seed=0):
    layer = Layer(device, seed)
    gen = torch.Generator(device=device).manual_seed(seed + 1)
    prompts = [50, 1, 77]
    n_req = len(prompts)
    kv = B.DeviceKV8.empty(24, HEADS, HEAD_DIM, PAGE, kind, device)
    pages = Pages(kv.n_pages, n_req, 16, device)
    adapter = [0, -1, 1]                       # request 1 has no adapter
    cached, worst = [0] * n_req, 0.0
    for t in range(steps + 1):
        new = prompts if t == 0 else [1] * n_req
        total = [c + n for c, n in zip(cached, new)]
        for r in range(n_req):
            pages.grow(r, total[r])
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device=device)  # noqa: E731
        start = ints([sum(new[:r]) for r in range(n_req + 1)])
        ids = ints([adapter[r] for r in range(n_req) for _ in range(new[r])])
        X = torch.randn(sum(new), D_MODEL, generator=gen, device=device).half()
        table = pages.device_table()
        q, y = step(layer, kv, X, ids, start, ints(cached), table, window, sinks)
        worst = max(worst, check(layer, kv, q, y, start, total, table, window, sinks))
        cached = total
        for r in range(n_req):
            pages.shrink(r, cached[r], window, sinks)
    print(f"{kind}: prompts of {prompts}, then {steps} tokens each; largest error "
          f"{worst:.2e} of the largest output; {len(pages.free)} of {kv.n_pages} pages free",
          flush=True)
    return worst


if __name__ == "__main__":
    for which in ("fp8", "int8"):
        main(which)
