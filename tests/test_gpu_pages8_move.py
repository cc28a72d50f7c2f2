"""Forking a batch of sequences on 8-bit pages and compacting their pool against
the oracle (oracle/pages8_oracle.py): every table, count and byte is equal."""
import numpy as np
import pytest
import torch

import oracle.pages8_oracle as Q
import compressed_composable_kv_gb300 as P
from compressed_composable_kv_gb300 import synth as S

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


class Pages:
    """A pool with bytes of all kinds, sequences of these lengths, the first
    `shared` pages of each taken from the sequence before it."""

    def __init__(self, lens, page=16, n_pages=None, layers=2, heads=2, d=64, width=None, shared=(), ahead=0, seed=0, scatter=True):
        rng = self.rng = np.random.default_rng(seed)
        self.g, self.page = S.Geometry(layers, 2 * heads, heads, d, 1e4), page
        counts = [max(0, -(-n // page)) + (ahead if n >= 0 else 0) for n in lens]
        share = [min(shared[i] if i < len(shared) else 0, counts[i], counts[i - 1] if i else 0, max(0, lens[i]) // page,
                     max(0, lens[i - 1]) // page if i else 0) for i in range(len(lens))]
        used = sum(counts) - sum(share)
        self.n_pages = n_pages = used + 5 if n_pages is None else n_pages
        ids = [int(x) for x in (rng.permutation(n_pages) if scatter else np.arange(n_pages))]
        self.width = max(1, max(counts) + 3) if width is None else width
        self.table = np.full((len(lens), self.width), -1, np.int32)
        self.refs = np.zeros(n_pages, np.int32)
        for b, c in enumerate(counts):
            row = [int(x) for x in self.table[b - 1, :share[b]]] if share[b] else []
            while len(row) < c:
                row.append(ids.pop())
            self.table[b, :c] = row
            self.refs[row] += 1
            self.table[b, c + 1:] = rng.integers(-9, 2 * n_pages, self.width)[c + 1:]   # behind the end: anything
        self.lens = np.asarray(lens, np.int32)
        shape = (layers, n_pages, heads, page, d)
        self.codes = [rng.integers(0, 256, shape, dtype=np.uint8) for _ in range(2)]
        self.scales = [np.exp2(rng.integers(-9, 9, shape[:3])).astype(np.float32) for _ in range(2)]
        self.upload()

    def upload(self):
        self.k8, self.v8 = (torch.from_numpy(c.copy()).cuda().view(E4) for c in self.codes)
        self.ks, self.vs = (torch.from_numpy(s.copy()).cuda() for s in self.scales)
        self.t_dev, self.r_dev, self.n_dev = _i32(self.table), _i32(self.refs), _i32(self.lens)

    def pool(self):
        return self.g, self.k8, self.v8, self.ks, self.vs

    def ws(self, batch):
        n = P.c2kv_pages8_plan_workspace_size(self.n_pages, max(batch, len(self.lens)), self.width)
        return torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")

    def fork(self, parent, room, stream=None):
        out = [torch.full((self.n_pages,), -55, dtype=torch.int32, device="cuda"),
               torch.full((len(parent), self.width), -55, dtype=torch.int32, device="cuda"),
               torch.full((len(parent),), -55, dtype=torch.int32, device="cuda")]
        P.c2kv_pages8_fork(*self.pool(), self.r_dev, self.t_dev, self.n_dev, _i32(parent), room, *out, self.ws(len(parent)), stream=stream)
        torch.cuda.synchronize()
        return out

    def check_fork(self, parent, room):
        want = Q.fork(self.refs, self.table, self.lens, parent, room, self.page)
        refs, table, n = self.fork(parent, room)
        if want is None:
            assert P.c2kv_device_error() == P.C2KV_EDEVICE
            assert all((x == -55).all() for x in (refs, table, n))
        else:
            assert P.c2kv_device_error() == P.C2KV_OK
            assert n.tolist() == want[2]
            assert table.tolist() == want[1]
            assert refs.tolist() == want[0]
            for src, dst, rows in want[3]:
                self.copy(src, dst, rows)
        self.check_bytes()
        return want

    def copy(self, src, dst, rows):
        for c, s in zip(self.codes, self.scales):
            c[:, dst, :, :rows] = c[:, src, :, :rows]
            s[:, dst] = s[:, src]

    def check_bytes(self):
        for dev, ref in ((self.k8, self.codes[0]), (self.v8, self.codes[1])):
            assert np.array_equal(dev.view(torch.uint8).cpu().numpy(), ref)
        for dev, ref in ((self.ks, self.scales[0]), (self.vs, self.scales[1])):
            assert np.array_equal(dev.cpu().numpy(), ref)

    def check_compact(self):
        want = Q.compact(self.refs, self.table)
        refs, table, moved = (torch.full(s, -55, dtype=torch.int32, device="cuda") for s in ((self.n_pages,), self.table.shape, (self.n_pages,)))
        P.c2kv_pages8_compact(*self.pool(), self.r_dev, self.t_dev, refs, table, moved, self.ws(1))
        torch.cuda.synchronize()
        if want is None:
            assert P.c2kv_device_error() == P.C2KV_EDEVICE
            assert all((x == -55).all() for x in (refs, table, moved))
        else:
            assert P.c2kv_device_error() == P.C2KV_OK
            assert refs.tolist() == want[0]
            assert table.tolist() == want[1]
            assert moved.tolist() == want[2]
            for src, dst in want[3]:
                self.copy(src, dst, self.page)
        self.check_bytes()
        return want


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("room", [0, 1, 40, 300])
def test_fork(page, d, room):
    """Places that go on, split, end and stay empty; lengths at and around the
    ends of pages."""
    lens = [0, 1, page - 1, page, page + 1, 2 * page, -1, 200, 133]
    p = Pages(lens, page, 200, d=d, width=40, shared=[0, 0, 0, 0, 1, 1, 0, 0, 1], seed=page + d + room)
    p.check_fork([8, 0, 8, -1, 2, 3, 3, 3, 6, 7, 4, 4, -5, 5, 5, 8, 1], room)


def test_fork_keeps_what_was_taken_ahead():
    """Pages behind the length go with the first child; room takes no more than it needs."""
    p = Pages([20, 33, 16, 0], 16, 40, ahead=3, seed=1)
    p.check_fork([1, 0, 1, 2, 3, 3], 30)
    p = Pages([20, 33, 16, 0], 16, 40, ahead=3, seed=2)
    p.check_fork([0, 1, 2, 3], 60)


def test_fork_ends_all_and_begins_none():
    p = Pages([100, 50, 17], 16, seed=3)
    want = p.check_fork([-1, -1], 10)
    assert sum(want[0]) == 0
    p = Pages([-1, -1], 16, 9, seed=4)
    p.check_fork([0, 1, -1, 1], 10)


def test_fork_takes_pages_that_the_call_gives_back():
    """A full pool: what ends makes room for what goes on."""
    p = Pages([64, 64, 30], 16, 10, width=12, seed=5, scatter=False)
    want = p.check_fork([2, 2, 2], 16)
    assert want is not None and len(want[3]) == 2


@pytest.mark.parametrize("free,ok", [(3, True), (2, False)])
def test_fork_of_too_few_free_pages_writes_nothing(free, ok):
    p = Pages([40, 30], 16, 5 + free, width=9, seed=6)
    want = p.check_fork([0, 0, 1, 1, 1], 0)
    assert (want is not None) == ok


def test_fork_of_bad_values_writes_nothing():
    def bad(change, parent=(0, 1), room=0, width=8):
        p = Pages([40, 30, -1], 16, 12, width=width, seed=7)
        change(p)
        p.upload()
        assert p.check_fork(list(parent), room) is None
        p.check_bytes()

    def entry(p, v):
        p.table[1, 1] = v

    bad(lambda p: entry(p, 12))
    bad(lambda p: entry(p, 1 << 30))
    bad(lambda p: entry(p, int(np.flatnonzero(p.refs == 0)[0])))
    bad(lambda p: p.refs.__setitem__(11, -1))
    bad(lambda p: p.lens.__setitem__(0, 49))
    bad(lambda p: None, parent=(0, 3))
    bad(lambda p: None, parent=(0, 1), room=100, width=4)
    bad(lambda p: p.table.__setitem__((1, 0), p.table[0, 0]), parent=(-1, -1))   # named more often than refs says


def test_fork_in_place():
    p = Pages([100, 50, 17, 64], 16, 60, shared=[0, 2], seed=8)
    parent = [1, 1, 3, -1]
    want = Q.fork(p.refs, p.table, p.lens, parent, 20, 16)
    P.c2kv_pages8_fork(*p.pool(), p.r_dev, p.t_dev, p.n_dev, _i32(parent), 20, p.r_dev, p.t_dev, p.n_dev, p.ws(4))
    torch.cuda.synchronize()
    assert P.c2kv_device_error() == P.C2KV_OK
    assert (p.r_dev.tolist(), p.t_dev.tolist(), p.n_dev.tolist()) == (want[0], want[1], want[2])
    for c in want[3]:
        p.copy(*c)
    p.check_bytes()


def test_fork_of_256_sequences_and_a_large_pool():
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(-1, 900, 256)]
    p = Pages(lens, 16, 30000, layers=1, heads=1, shared=[int(x) for x in rng.integers(0, 30, 256)], seed=9)
    p.check_fork([int(x) for x in rng.integers(-20, 256, 256)], 70)


def test_beams_over_many_steps():
    """Parents and lengths as a search has them, in place, step by step: the
    oracle follows, and no page is lost."""
    p = Pages([37] * 4, 16, 80, width=20, shared=[0, 2, 2, 2], seed=10)
    ws = p.ws(4)
    for step in range(60):
        parent = [int(x) for x in p.rng.integers(0, 4, 4)]
        want = Q.fork(p.refs, p.table, p.lens, parent, 1, 16)
        P.c2kv_pages8_fork(*p.pool(), p.r_dev, p.t_dev, p.n_dev, _i32(parent), 1, p.r_dev, p.t_dev, p.n_dev, ws)
        P.c2kv_seq_advance(p.n_dev, 1)
        p.refs, p.table, lens, copies = np.asarray(want[0]), np.asarray(want[1]), want[2], want[3]
        for c in copies:
            p.copy(*c)
        p.lens = np.asarray(lens) + 1
        held = {int(e) for row in p.table for e in row if e >= 0}
        assert held == set(np.flatnonzero(p.refs))
    torch.cuda.synchronize()
    assert P.c2kv_device_error() == P.C2KV_OK
    assert np.array_equal(p.r_dev.cpu().numpy(), p.refs) and np.array_equal(p.t_dev.cpu().numpy(), p.table)
    p.check_bytes()


# ------------------------------------------------------------------ compact

@pytest.mark.parametrize("page,d", [(16, 64), (32, 128), (64, 64), (128, 128)])
@pytest.mark.parametrize("n_pages", [29, 64, 500])
def test_compact(page, d, n_pages):
    p = Pages([3 * page, 1, 5 * page - 1, -1, 7 * page + 1], page, n_pages, d=d, shared=[0, 0, 1, 0, 2], seed=n_pages + d)
    p.check_compact()


def test_compact_of_all_of_none_and_of_what_is_in_front():
    p = Pages([64, 80], 16, 9, seed=11)
    assert p.check_compact()[3] == []           # every page in use
    p = Pages([-1, -1], 16, 9, seed=12)
    assert p.check_compact()[3] == []           # none
    p = Pages([64, 80], 16, 33, seed=13, scatter=False)
    p.check_compact()
    p = Pages([64], 16, 1000, seed=14)          # pages that no sequence of the table names
    p.refs[999], p.refs[3] = 2, 1
    p.upload()
    p.check_compact()


def test_compact_of_a_large_pool():
    rng = np.random.default_rng(15)
    p = Pages([int(x) for x in rng.integers(-1, 900, 256)], 16, 20000, layers=1, heads=1, seed=15)
    p.check_compact()


def test_compact_of_bad_values_writes_nothing():
    for change in (lambda p: p.table.__setitem__((0, 1), 40), lambda p: p.table.__setitem__((0, 1), int(np.flatnonzero(p.refs == 0)[0])),
                   lambda p: p.refs.__setitem__(39, -2)):
        p = Pages([40, 30], 16, 40, seed=16)
        change(p)
        p.upload()
        assert p.check_compact() is None


def test_compact_in_place_without_the_map():
    p = Pages([100, 50, 17, 64], 16, 90, shared=[0, 2], seed=17)
    want = Q.compact(p.refs, p.table)
    P.c2kv_pages8_compact(*p.pool(), p.r_dev, p.t_dev, p.r_dev, p.t_dev, None, p.ws(4))
    torch.cuda.synchronize()
    assert P.c2kv_device_error() == P.C2KV_OK
    assert (p.r_dev.tolist(), p.t_dev.tolist()) == (want[0], want[1])
    for src, dst in want[3]:
        p.copy(src, dst, 16)
    p.check_bytes()


@pytest.mark.parametrize("batch,n_pages", [(32, 2048), (33, 2048), (32, 2049), (1, 2047), (33, 2049)])
def test_few_and_many_pages(batch, n_pages):
    """The plan is made by one block of threads or by several: both sides of the border."""
    rng = np.random.default_rng(batch + n_pages)
    lens = [int(x) for x in rng.integers(0, 600, batch)]
    shared = [int(x) for x in rng.integers(0, 8, batch)]
    p = Pages(lens, 16, n_pages, layers=1, heads=1, width=60, shared=shared, seed=batch)
    p.check_fork([int(x) for x in rng.integers(-2, batch, 40)], 33)
    p = Pages(lens, 16, n_pages, layers=1, heads=1, shared=shared, seed=batch)
    p.check_compact()


def test_fork_and_compact_in_a_graph_and_on_another_stream():
    p = Pages([100, 50, 17, 64], 16, 90, seed=18)
    side = torch.cuda.Stream()
    first = p.fork([0, 0, 1, 1], 5)
    second = p.fork([0, 0, 1, 1], 5, stream=side)
    assert all(torch.equal(x, y) for x, y in zip(first, second))
    parent, out, ws = _i32([0, 0, 1, 1]), [torch.empty_like(x) for x in first], p.ws(4)
    out2 = [torch.empty_like(out[0]), torch.empty_like(out[1]), torch.empty_like(out[0])]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.c2kv_pages8_fork(*p.pool(), p.r_dev, p.t_dev, p.n_dev, parent, 5, *out, ws)
        P.c2kv_pages8_compact(*p.pool(), out[0], out[1], *out2, ws)
    want = Q.fork(p.refs, p.table, p.lens, [0, 0, 1, 1], 5, 16)
    w2 = Q.compact(want[0], want[1])
    graph.replay()
    torch.cuda.synchronize()
    assert P.c2kv_device_error() == P.C2KV_OK
    assert [x.tolist() for x in out] == [want[0], want[1], want[2]]
    assert [x.tolist() for x in out2] == [w2[0], w2[1], w2[2]]
    for c in want[3]:
        p.copy(*c)
    for src, dst in w2[3]:
        p.copy(src, dst, 16)
    p.check_bytes()
