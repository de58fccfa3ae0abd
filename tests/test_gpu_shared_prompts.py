"""The calls for shared prompts together, as a server uses them: prompts are cached, each is forked
to its beams, and every step makes the pages of the next token (kv8_tables), appends it, attends
over the shared prompt (kv8_prefix_attention), picks the next beams (beam_select) and gives the
rows to them (kv8_reorder, kv8_copy_pages), in two layers' caches over one table.

The reference keeps a cache of its own for every beam, without any sharing, and copies it whole
when beams change places: codes have to be equal, outputs within the attention's bound."""
import numpy as np
import pytest
import torch

from dictionary_factored_sparse_amd import binding as B
from tests import pages_ref as PR
from tests import serving_ref as R
from tests.gpu_helpers import DEV, say
from tests.test_gpu_beam import check as check_beams
from tests.test_gpu_serving import within

pytestmark = pytest.mark.gpu
HEADS, GROUP, DIM, PAGE, VOCAB, LAYERS = 2, 2, 64, 16, 331, 2
COLS = HEADS * DIM


def ints(v):
    return torch.tensor(np.asarray(v, np.int32), device=DEV)


class Toy:
    """Something that makes keys, values, queries and logits of tokens and attention outputs."""

    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
        self.k, self.v = [r(VOCAB, COLS).half() for _ in range(2)], [r(VOCAB, COLS).half()
                                                                     for _ in range(2)]
        self.q = [r(VOCAB, GROUP * COLS).half() for _ in range(2)]
        self.out = (0.8 * r(GROUP * COLS, VOCAB)).half()

    def logits(self, o):
        return sum(o).half() @ self.out


class Server:
    def __init__(self, kind, prompts, width, n_pages=60, seed=0):
        rng = np.random.default_rng(seed)
        self.toy, self.width, self.n = Toy(seed), width, len(prompts)
        self.kvs = [B.DeviceKV8.empty(n_pages, HEADS, DIM, PAGE, kind, DEV) for _ in range(LAYERS)]
        self.refs = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
        rows = self.n * width
        self.tables = [torch.full((rows, 12), -1, dtype=torch.int32, device=DEV) for _ in range(2)]
        self.batch = B.DeviceBatch.empty(rows, rows, DEV)
        self.one = torch.ones(rows, dtype=torch.int32, device=DEV)
        self.cached = torch.zeros(rows, dtype=torch.int32, device=DEV)
        self.tokens = torch.zeros(rows, dtype=torch.int64, device=DEV)
        self.score = torch.full((rows,), -np.inf, device=DEV)
        self.score[::width] = 0.0
        self.done = torch.zeros(rows, dtype=torch.int32, device=DEV)
        self.ws_att = B.kv8_prefix_attention_workspace(self.kvs[0], rows, rows, HEADS * GROUP, DEV)
        self.ws_beam = B.beam_workspace(self.n, width, VOCAB, DEV)
        self.ws_reorder = B.kv8_reorder_workspace(rows, DEV)
        self.groups = ints(width * np.arange(self.n + 1))
        self.shared = ints([t // PAGE * PAGE for t in prompts])
        # the prompts, and one row for each beam
        table = torch.full((self.n, 12), -1, dtype=torch.int32, device=DEV)
        zero = torch.zeros(self.n, dtype=torch.int32, device=DEV)
        b = B.kv8_tables(self.refs, PAGE, zero, ints(prompts), table, n_tok=sum(prompts))
        text = torch.from_numpy(rng.integers(0, VOCAB, sum(prompts))).to(DEV)
        assert torch.equal(b.tok_pos, torch.cat([torch.arange(t) for t in prompts]).int().to(DEV))
        for i, kv in enumerate(self.kvs):
            B.kv8_append(kv, self.toy.k[i][text], self.toy.v[i][text], b.tok_start, zero, table)
        length, src, dst, missing = B.kv8_reorder(
            self.refs, PAGE, table, b.length, ints(np.repeat(np.arange(self.n), width)),
            self.tables[0])
        B.kv8_copy_pages(self.kvs, src, dst, length)
        assert missing.item() == 0 and b.missing.item() == 0
        self.cached.copy_(length)
        first = np.cumsum(prompts) - 1
        self.tokens.copy_(text[torch.from_numpy(first).to(DEV)].repeat_interleave(width))
        self.text, self.prompts, self.now = text.cpu().numpy(), prompts, 0

    def step(self):
        """One token for every beam, on the current stream; nothing of it waits."""
        t, s = self.tables[self.now], self
        b = B.kv8_tables(s.refs, PAGE, s.cached, s.one, t, s.batch)
        o = []
        for i, kv in enumerate(s.kvs):
            B.kv8_append(kv, s.toy.k[i][s.tokens], s.toy.v[i][s.tokens], b.tok_start, s.cached, t)
            o.append(B.kv8_prefix_attention(kv, s.toy.q[i][s.tokens], b.tok_start, b.length, t,
                                            s.groups, s.shared, HEADS * GROUP,
                                            odtype=torch.float32, ws=s.ws_att))
        logits = s.toy.logits(o)
        parent, token, score, done = B.beam_select(logits, s.score, s.width, eos=3, done=s.done,
                                                   ws=s.ws_beam)
        parent = torch.where(token < 0, torch.arange(len(token), device=DEV), parent).int()
        length, src, dst, missing = B.kv8_reorder(s.refs, PAGE, t, b.length, parent,
                                                  s.tables[1 - s.now], ws=s.ws_reorder)
        B.kv8_copy_pages(s.kvs, src, dst, length)
        seen = dict(o=o, logits=logits, was=s.score.clone(), ended=s.done.clone(), parent=parent,
                    token=token, score=score, done=done, missing=missing, lost=b.missing)
        s.cached.copy_(length)
        s.tokens.copy_(token.clamp(min=0))
        s.score.copy_(score)
        s.done.copy_(done)
        s.now = 1 - s.now
        return seen


class Mirror:
    """The beams' caches in numpy, one for each."""

    def __init__(self, server, kind):
        s, self.kind = server, kind
        rows, per = s.n * s.width, s.tables[0].shape[1]
        self.rows, self.per = rows, per
        self.table = np.arange(rows * per).reshape(rows, per)
        self.caches = []
        for i in range(LAYERS):
            c = [np.zeros((rows * per, HEADS, PAGE, DIM), np.uint8),
                 np.zeros((rows * per, HEADS, DIM, PAGE), np.uint8),
                 np.zeros((rows * per, HEADS), np.float32), np.zeros((rows * per, HEADS), np.float32)]
            starts = np.concatenate([[0], np.cumsum(s.prompts)])
            for r in range(rows):
                t = s.text[starts[r // s.width]:starts[r // s.width + 1]]
                R.append(*c, kind, s.toy.k[i].float().cpu().numpy()[t],
                         s.toy.v[i].float().cpu().numpy()[t], [0, len(t)], [0], self.table[r:r + 1],
                         PAGE)
            self.caches.append(c)
        self.length = np.repeat(s.prompts, s.width)

    def append(self, i, K, V):
        R.append(*self.caches[i], self.kind, K, V, np.arange(self.rows + 1), self.length, self.table,
                 PAGE)

    def attend(self, i, Q):
        return R.attention(*self.caches[i], self.kind, Q, np.arange(self.rows + 1), self.length + 1,
                           self.table, HEADS * GROUP, DIM ** -0.5, 0, 0, "f32")

    def reorder(self, parent):
        self.length = (self.length + 1)[parent]
        for c in self.caches:
            for j, a in enumerate(c):
                b = a.reshape(self.rows, self.per, *a.shape[1:])[parent]
                c[j] = b.reshape(a.shape).copy()

    def same(self, server):
        table = server.tables[server.now].cpu().numpy()
        for i, kv in enumerate(server.kvs):
            k, v, ks, vs = (t.cpu().numpy() for t in (kv.k, kv.v, kv.kscale, kv.vscale))
            for r in range(self.rows):
                for p in range(-(-self.length[r] // PAGE)):
                    m, own, pg = min(PAGE, self.length[r] - p * PAGE), self.table[r, p], table[r, p]
                    c = self.caches[i]
                    assert np.array_equal(k[pg, :, :m], c[0][own, :, :m]), (i, r, p)
                    assert np.array_equal(v[pg, :, :, :m], c[1][own, :, :, :m]), (i, r, p)
                    assert np.array_equal(ks[pg], c[2][own]) and np.array_equal(vs[pg], c[3][own])


@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_beams_over_shared_prompts(kind):
    s = Server(kind, [37, 80], 3)
    m = Mirror(s, kind)
    m.same(s)
    moved = forks = 0
    for t in range(36):
        say(f"case: beams over shared prompts, {kind}, step {t}")
        tok = s.tokens.cpu().numpy()
        before = m.length.copy()
        seen = s.step()
        for i in range(LAYERS):
            m.append(i, s.toy.k[i].float().cpu().numpy()[tok], s.toy.v[i].float().cpu().numpy()[tok])
            ref, bound, _ = m.attend(i, s.toy.q[i].double().cpu().numpy()[tok])
            within(seen["o"][i], ref, bound, f"step {t} layer {i}")
        parent = seen["parent"].cpu().numpy()
        check_beams(seen["logits"].float().cpu().numpy(), seen["was"].cpu().numpy(), 3, 3,
                    seen["ended"].cpu().numpy(),
                    got=(torch.where(seen["token"] < 0, seen["parent"] // 3 * 3, seen["parent"]),
                         seen["token"], seen["score"], seen["done"]))
        m.reorder(parent)
        m.same(s)
        assert seen["missing"].item() == 0 and seen["lost"].item() == 0
        assert np.array_equal(s.cached.cpu().numpy(), m.length) and (m.length >= before).all()
        table = s.tables[s.now].cpu().numpy()
        assert np.array_equal(s.refs.cpu().numpy(), PR.counts(s.refs.shape[0], table))
        moved += int((parent != np.arange(6)).sum())
        forks += 6 - len(set(parent.tolist()))
    assert moved > 20 and forks > 10
    B.kv8_release(s.refs, s.tables[s.now])
    assert not s.refs.any() and (s.tables[s.now] == -1).all()


def test_a_captured_step_follows_the_beams():
    """Two steps (from one table to the other and back) captured once and replayed: the same as
    eager ones, with eager work and waits between the replays."""
    a, b = Server("fp8", [37, 80, 5], 4, n_pages=90), Server("fp8", [37, 80, 5], 4, n_pages=90)
    state = lambda s: [s.refs, s.tables[s.now], s.cached, s.tokens, s.score, s.done] + [  # noqa: E731
        t for kv in s.kvs for t in (kv.kscale, kv.vscale)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):          # first calls, outside of the capture
        b.step()
        b.step()
    side.synchronize()
    a.step()
    a.step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        b.step()
        b.step()
    junk = torch.zeros(1 << 20, device=DEV)
    for i in range(12):
        say(f"case: captured steps, replay {i}")
        g.replay()
        junk.add_(1.0)
        torch.cuda.synchronize()
        a.step()
        a.step()
        for x, y in zip(state(a), state(b)):
            assert torch.equal(x, y), i
    assert (junk == 12).all()


def test_on_a_stream_given_by_argument():
    """Outputs and workspaces that the calls make are in the order of that stream."""
    rng = np.random.default_rng(2)
    kv = B.DeviceKV8.empty(40, HEADS, DIM, PAGE, "int8", DEV)
    kv.k.copy_(torch.from_numpy(rng.integers(0, 256, kv.k.shape).astype(np.uint8)))
    kv.v.copy_(torch.from_numpy(rng.integers(0, 256, kv.v.shape).astype(np.uint8)))
    kv.kscale.fill_(0.01)
    kv.vscale.fill_(0.01)
    q = torch.randn(4, GROUP * COLS, device=DEV).half()
    logits, score = torch.randn(8, 5000, device=DEV), -torch.rand(8, device=DEV)
    big = torch.randn(4096, 4096, device=DEV).half()

    def calls(stream):
        refs = torch.zeros(40, dtype=torch.int32, device=DEV)
        table = torch.full((4, 8), -1, dtype=torch.int32, device=DEV)
        out = torch.full((4, 8), -1, dtype=torch.int32, device=DEV)
        cached, new, ones = ints([0, 0, 0, 0]), ints([50, 100, 37, 96]), ints([1, 1, 1, 1])
        torch.cuda.synchronize()
        if stream is not None:
            junk = [torch.full((1 << 24,), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]
            torch.cuda.synchronize()
            del junk                   # what the allocator gives next is not zero
            for _ in range(10):
                big @ big
        b = B.kv8_tables(refs, PAGE, cached, new, table, n_tok=300, stream=stream)
        got = B.kv8_reorder(refs, PAGE, table, b.length, ints([1, 1, 0, 3]), out, stream=stream)
        B.kv8_copy_pages([kv], got[1], got[2], got[0], stream=stream)
        o = B.kv8_prefix_attention(kv, q, ints(range(5)), got[0], out, ints([0, 2, 4]),
                                   ints([64, 0]), HEADS * GROUP, stream=stream)
        beams = B.beam_select(logits, score, 4, stream=stream)
        B.kv8_release(refs, out, ones, stream=stream)
        (torch.cuda.current_stream() if stream is None else stream).synchronize()
        return [b.tok_start, b.tok_pos, b.slot, *got, o, *beams, refs, out]

    k0, v0 = kv.k.clone(), kv.v.clone()
    want = calls(None)
    side = torch.cuda.Stream()
    for i in range(3):
        say(f"case: shared prompts on a stream given by argument, round {i}")
        kv.k.copy_(k0)
        kv.v.copy_(v0)
        for x, y in zip(want, calls(side)):
            assert torch.equal(x, y)


def test_an_input_let_go_of_is_kept_for_its_stream():
    """What a call on another stream reads is not handed out again before that call has run."""
    say("case: temporary inputs on a stream given by argument")
    table, length = ints(np.arange(32).reshape(4, 8)), ints([50, 100, 37, 96])
    refs, out = ints([1] * 40), ints(np.full((4, 8), -1))
    big = torch.randn(4096, 4096, device=DEV).half()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            big @ big
    got = B.kv8_reorder(refs, PAGE, table, length, ints([1, 1, 0, 3]), out, stream=side)
    others = [ints([3, 3, 3, 3]) for _ in range(8)]
    torch.cuda.synchronize()
    assert got[0].tolist() == [100, 100, 50, 96] and len(others) == 8


def test_two_streams_at_once():
    """Steps of two servers on streams of their own, each with its own workspaces, side by side."""
    mix = [Server("fp8", [37, 80], 4, n_pages=90), Server("int8", [100, 5, 64], 5, n_pages=140)]
    alone = [Server("fp8", [37, 80], 4, n_pages=90), Server("int8", [100, 5, 64], 5, n_pages=140)]
    say("case: two streams at once")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, st in zip(mix, streams):
            with torch.cuda.stream(st):
                s.step()
    torch.cuda.synchronize()
    for s in alone:
        for _ in range(20):
            s.step()
    for a, b in zip(mix, alone):
        assert torch.equal(a.refs, b.refs) and torch.equal(a.tables[a.now], b.tables[b.now])
        assert torch.equal(a.cached, b.cached) and torch.equal(a.tokens, b.tokens)
        assert torch.equal(a.score, b.score) and torch.equal(a.done, b.done)
