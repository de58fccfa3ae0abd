"""How the serving calls are made: on a stream given by argument, with one workspace kept for
calls of many sizes."""
import numpy as np
import pytest
import torch

from dictionary_factored_sparse_amd import binding as B
from tests.gpu_helpers import DEV, say
from tests.test_gpu_serving import Cache, ints, make_adapters

pytestmark = pytest.mark.gpu


def halves(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float16)).to(DEV)


def test_calls_on_a_stream_given_by_argument():
    """Workspaces and outputs that the calls make are in the order of that stream, whatever the
    current one is busy with."""
    rng = np.random.default_rng(1)
    lengths = [700, 33, 2000]
    c = Cache(rng, "fp8", 2, 128, 64, lengths)
    ad, _ = make_adapters(rng, 5, 64, 512, 256, [64, 8, 33, 5, 64])
    X, ids, Q = halves(rng, 300, 512), ints(rng.integers(-1, 5, 300)), halves(rng, 3, 512)
    K, V = halves(rng, 3, 256), halves(rng, 3, 256)
    start, cached, length = ints([0, 1, 2, 3]), ints(np.array(lengths) - 1), ints(lengths)
    Y = B.dict_adapter_forward(X, ad, ids)
    B.kv8_append(c.kv, K, V, start, cached, c.tab)
    O = B.kv8_attention(c.kv, Q, start, length, c.tab, 4)
    big = torch.randn(4096, 4096, device=DEV).half()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for i in range(4):
        say(f"case: stream given by argument, round {i}")
        junk = [torch.full((1 << 24,), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]
        torch.cuda.synchronize()
        del junk                       # what the current stream's allocator gives next is not zero
        for _ in range(10):
            big @ big
        y = B.dict_adapter_forward(X, ad, ids, stream=side)
        B.kv8_append(c.kv, K, V, start, cached, c.tab, stream=side)
        o = B.kv8_attention(c.kv, Q, start, length, c.tab, 4, stream=side)
        side.synchronize()
        assert torch.equal(y, Y) and torch.equal(o, O)


def test_one_adapter_workspace_for_every_smaller_batch():
    """A workspace for 9000 tokens, full of NaN, serves smaller batches in any order."""
    rng = np.random.default_rng(2)
    for n, r_max in ((3, 32), (24, 64), (300, 8)):
        ad, _ = make_adapters(rng, n, r_max, 1096, 72, rng.integers(1, r_max + 1, n))
        X, ids = halves(rng, 9000, 1096), ints(rng.integers(-1, n, 9000))
        ws = B.adapter_workspace(9000, ad, DEV)
        for T in (9000, 5, 300, 1, 8192, 64, 191, 192, 256, 257, 1024, 8193):
            say(f"case: adapters, one workspace, n={n} T={T}")
            ws.fill_(0xFF)
            y = B.dict_adapter_forward(X[:T], ad, ids[:T], ws=ws)
            assert torch.equal(y, B.dict_adapter_forward(X[:T], ad, ids[:T]))
            assert torch.isfinite(y).all()


def test_one_attention_workspace_for_every_smaller_batch():
    """A workspace for 12 requests and 700 tokens serves decode batches, drafts, prompts and many
    kinds of batches between, in any order; only its first 64 KiB are cleared, once."""
    rng = np.random.default_rng(3)
    lengths = [900, 700, 64, 1, 130, 333, 17, 500, 250, 80, 40, 700]
    c = Cache(rng, "int8", 2, 64, 32, lengths)
    H = 6
    ws = B.kv8_attention_workspace(c.kv, 12, 700, H, DEV)
    ws[65536:] = 0xFF
    Q = halves(rng, 700, H * 64)
    for r0, r1, new in ((0, 12, 1), (0, 1, 700), (0, 12, 7), (3, 4, 1), (0, 2, 300), (7, 12, 3),
                        (0, 1, 11), (0, 6, 60), (0, 1, 5), (2, 3, 64), (0, 12, 1)):
        n = np.minimum(new, lengths[r0:r1])
        say(f"case: attention, one workspace, requests {r0}..{r1 - 1}, new {n.tolist()}")
        args = (c.kv, Q[:n.sum()], ints(np.concatenate([[0], np.cumsum(n)])), ints(lengths[r0:r1]),
                c.tab[r0:r1], H)
        o = B.kv8_attention(*args, ws=ws)
        assert not ws[:65536].any()
        assert torch.equal(o, B.kv8_attention(*args)) and torch.isfinite(o).all()
