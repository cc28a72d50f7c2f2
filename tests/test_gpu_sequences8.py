"""Sequences on shared 8-bit pages from the composed requests on: answers forked,
a further question taken in as a chunk, tokens decoded, beams moved, answers ended,
the pool compacted, against the fp64 oracle's pages all along the way.  Bars as in
test_gpu_chunk8.py and test_gpu_pages8.py."""
import numpy as np
import pytest
import torch

import oracle.pages8_oracle as Q
import compressed_composable_kv_gb300 as P
from compressed_composable_kv_gb300 import synth as S
from gpu_util import Scenario, to_bits, upload
from test_gpu_pages8 import _dev, _f64, _rotate, _round_key, _values

pytestmark = pytest.mark.gpu


class World:
    """Prefilled requests with spare pages, their sequences, and the oracle's pool."""

    def __init__(self, g, page, batch=2, q_len=9, spare=60, steps=80):
        self.g, self.page = g, page
        specs = [(i, 400 + 300 * i, 100 + 75 * i) for i in range(3)]
        requests = [([i % 3, (i + 1) % 3][: 1 + i % 2], None) for i in range(batch)]
        self.sc = Scenario(g, 4, specs, requests, q_len=q_len, decode_steps=steps)
        self.rb = rb = P.RequestBatch(self.sc.store, g, self.sc.reqs, 4, q_len, steps, page8=page, spare_pages=spare)
        dev = upload(S.make_step_inputs(S.Workload("sequences8", g, 4, batch, q_len, 1, seed=5)))
        rb.compose()
        for l in range(g.n_layers):
            rb.prefill(l, dev["q_pre"][l], dev["kq_pre"][l], dev["vq"][l], torch.empty_like(dev["q_pre"][l]))
        rb.fill_pages8()
        torch.cuda.synchronize()
        self.rng = np.random.default_rng(page)
        self.codes = [x.view(torch.uint8).cpu().numpy().copy() for x in (rb.k8, rb.v8)]
        self.scales = [x.cpu().numpy().copy() for x in (rb.k_scale, rb.v_scale)]
        need = [-(-(n + q_len) // page) for n in rb.n_slots]
        table = rb.page_table.cpu().numpy()
        self.table = [list(row[:c]) + [-1] * (len(row) - c) for row, c in zip(table, need)]
        self.refs = [0] * rb.k8.shape[1]
        for row in self.table:
            for p in row:
                if p >= 0:
                    self.refs[p] += 1
        self.lens = [n + q_len for n in rb.n_slots]
        self.first = [lt + q_len - n for lt, n in zip(rb.l_tot, self.lens)]   # a row's position, less the row

    def fork(self, parents, room):
        self.refs, self.table, lens, copies = Q.fork(self.refs, self.table, self.lens, parents, room, self.page)
        self.first = [self.first[p] if p >= 0 else 0 for p in parents]
        self.lens = lens
        for src, dst, rows in copies:
            self.copy(src, dst, rows)

    def copy(self, src, dst, rows):
        for c, s in zip(self.codes, self.scales):
            c[:, dst, :, :rows] = c[:, src, :, :rows]
            s[:, dst] = s[:, src]

    def compact(self):
        self.refs, self.table, _, moves = Q.compact(self.refs, self.table)
        for src, dst in moves:
            self.copy(src, dst, self.page)

    def check(self, seqs, what):
        torch.cuda.synchronize()
        assert P.c2kv_device_error() == P.C2KV_OK, what
        assert seqs.page_table.tolist() == [list(map(int, r)) for r in self.table], what
        assert seqs.refs.tolist() == [int(r) for r in self.refs], what
        assert seqs.n_cached_dev.tolist() == list(self.lens), what
        for dev, scale, c, s in ((seqs.k8, seqs.k_scale, self.codes[0], self.scales[0]), (seqs.v8, seqs.v_scale, self.codes[1], self.scales[1])):
            codes, scales = dev.view(torch.uint8).cpu().numpy(), scale.cpu().numpy()
            for b, n in enumerate(self.lens):
                for l in range(self.g.n_layers if n > 0 else 0):
                    a, r = (Q.held(x[l], y[l], self.page, self.table[b], n) for x, y in ((codes, scales), (c, s)))
                    assert np.array_equal(a, r), f"{what}: layer {l} sequence {b}: {int((a != r).sum())} held values differ"

    def tokens(self, seqs, new, call, parts, what, stream=None):
        """new[b] tokens of each sequence through every layer by call(l, q, k, v, out),
        on the device and in the oracle; the lengths are the oracle's to advance."""
        g, t = self.g, max(new)
        b = len(self.lens)
        for l in range(g.n_layers):
            q = _values(self.rng, (b, t, g.n_q_heads, g.head_dim))
            k, v = (_values(self.rng, (b, t, g.n_kv_heads, g.head_dim)) for _ in range(2))
            out = torch.full((b, t, g.n_q_heads, g.head_dim), -7.0, dtype=torch.bfloat16, device="cuda")
            call(l, _dev(q), _dev(k), _dev(v), out)
            torch.cuda.synchronize()
            got = out.float().cpu().numpy().astype(np.float64)
            for s, (n, c) in enumerate(zip(self.lens, new)):
                if n < 0 or c == 0:
                    assert (got[s] == -7.0).all(), what
                    continue
                pos = self.first[s] + n + np.arange(c)
                kr = _round_key(_rotate(g, _f64(k[s, :c]), pos))
                for kv, x in ((0, kr), (1, _f64(v[s, :c]))):
                    Q.put(self.codes[kv][l], self.scales[kv][l], self.page, self.table[s], n, x.transpose(1, 0, 2))
                K, V = (Q.held(self.codes[i][l], self.scales[i][l], self.page, self.table[s], n + c) for i in (0, 1))
                qr = _rotate(g, _f64(q[s, :c]), pos)
                ref = Q.attend_chunk(qr, K, V, n)
                ds = parts * np.abs(qr).max() * np.abs(K).sum(-1).max() / np.sqrt(g.head_dim)
                tol = 2.0 ** -8 * np.abs(ref) + (2 * ds + 2.0 ** -11 + 2.0 ** -31 * (n + c)) * np.abs(V).max()
                assert (np.abs(got[s, :c] - ref) <= tol).all(), f"{what}: layer {l} sequence {s}"
                assert (got[s, c:] == -7.0).all(), what

    def chunk(self, seqs, new, what):
        t = max(new)
        n_new = None if all(n == t for n in new) else torch.tensor(new, dtype=torch.int32, device="cuda")
        self.tokens(seqs, new, lambda l, q, k, v, out: seqs.chunk(l, q, k, v, out, n_new), 2.0 ** -11, what)
        seqs.advance(n=t if n_new is None else n_new)
        self.lens = [n + c if n >= 0 else n for n, c in zip(self.lens, new)]

    def decode(self, seqs, steps, what):
        for _ in range(steps):
            def call(l, q, k, v, out):
                seqs.decode(l, q[:, 0].contiguous(), k[:, 0].contiguous(), v[:, 0].contiguous(), out[:, 0])
            self.tokens(seqs, [1 if n >= 0 else 0 for n in self.lens], call, 2.0 ** -14, what)
            seqs.advance()
            self.lens = [n + 1 if n >= 0 else n for n in self.lens]


@pytest.mark.parametrize("d,group,page", [(128, 4, 64), (128, 5, 16), (64, 2, 32), (64, 8, 128)])
def test_answers_questions_beams_and_a_compacted_pool(d, group, page):
    w = World(S.Geometry(2, 2 * group, 2, d, 5.0e5), page)
    seqs = w.rb.answers(3, room=20)
    w.fork([0, 0, 0, 1, 1, 1], 20)
    w.check(seqs, "answers")
    w.decode(seqs, 3, "first tokens")
    w.check(seqs, "first tokens")
    w.chunk(seqs, [7, 1, 0, 17, 5, 2], "a further question")
    w.check(seqs, "a further question")
    parents = [1, 1, -1, 3, 5, 3]
    seqs.fork(torch.tensor(parents, dtype=torch.int32, device="cuda"), 30)
    w.fork(parents, 30)
    w.check(seqs, "beams")
    w.decode(seqs, 2, "beams")
    w.chunk(seqs, [9, 28, 0, 1, 28, 3], "drafts")
    w.check(seqs, "drafts")
    seqs.fork([4, -1, 0], 5)
    w.fork([4, -1, 0], 5)
    seqs.compact()
    w.compact()
    w.check(seqs, "compacted")
    used = sum(r > 0 for r in w.refs)
    assert all(r > 0 for r in seqs.refs[:used].tolist()) and used < len(w.refs)
    w.decode(seqs, 3, "compacted")
    w.check(seqs, "at the end")
    w.sc.close()


def test_decoder_model_over_sequences():
    """DecoderModel steps over forked answers: the same bits for answers that share all
    they have seen, whatever pages they are on."""
    g = S.Geometry(2, 8, 2, 128, 5.0e5)
    w = World(g, 32)
    seqs = w.rb.answers(2, room=8)
    shape = S.ModelShape(256, 512, 512, 1e-5)
    rng = np.random.default_rng(0)

    def weight(*size):
        return torch.from_numpy(rng.standard_normal(size).astype(np.float32) * size[-1] ** -0.5).to(torch.bfloat16).cuda()

    nq, nkv = 8 * 128, 2 * 128
    layers = [dict(attn_norm=torch.ones(256, dtype=torch.bfloat16, device="cuda"), qkv=weight(nq + 2 * nkv, 256), o=weight(256, nq),
                   mlp_norm=torch.ones(256, dtype=torch.bfloat16, device="cuda"), gate_up=weight(1024, 256), down=weight(256, 512))
              for _ in range(2)]
    model = P.DecoderModel(g, shape, dict(layers=layers), seqs.batch)
    x = weight(2, 256)
    for _ in range(4):
        model.x.copy_(x.repeat_interleave(2, 0))
        model.decode_step(seqs)
        torch.cuda.synchronize()
        assert P.c2kv_device_error() == P.C2KV_OK
        assert torch.equal(model.x[0], model.x[1]) and torch.equal(model.x[2], model.x[3])
        assert not torch.equal(model.x[0], model.x[2]) and torch.isfinite(model.x.float()).all()
        x = model.x[[0, 2]].clone()
    assert seqs.n_cached_dev.tolist() == [n + 4 for n in w.lens for _ in range(2)]
    w.sc.close()


def test_steps_on_another_stream_and_replayed():
    """Chunk, decode and advance captured once and replayed on a stream of their own."""
    g = S.Geometry(2, 8, 2, 128, 5.0e5)
    res = []
    for captured in (False, True):
        w = World(g, 16, spare=90)
        side = torch.cuda.Stream()
        seqs = w.rb.answers(2, room=40, stream=side)
        q = _dev(_values(w.rng, (4, 5, 8, 128)))
        k, v = (_dev(_values(w.rng, (4, 5, 2, 128))) for _ in range(2))
        o, o1 = torch.zeros_like(q), torch.zeros((2, 4, 8, 128), dtype=torch.bfloat16, device="cuda")
        q1, k1, v1 = (x[:, 0].contiguous() for x in (q, k, v))
        side.synchronize()
        torch.cuda.synchronize()

        def step():
            for l in range(2):
                seqs.chunk(l, q, k, v, o, stream=side)
            seqs.advance(side, 5)
            for l in range(2):
                seqs.decode(l, q1, k1, v1, o1[l], side)
            seqs.advance(side)

        with torch.cuda.stream(side):
            step()
            if captured:
                side.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    step()
                graph.replay()
                graph.replay()
            else:
                step()
                step()
        torch.cuda.synchronize()
        assert P.c2kv_device_error() == P.C2KV_OK
        res.append((o.clone(), o1.clone(), seqs.n_cached_dev.clone()))
        w.sc.close()
    for a, b in zip(*res):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n", [40, 250])
def test_a_pool_without_enough_pages_says_so(n):
    """All places go on with request 0: what request 1 gives back suffices for 40 of
    them, not for 250, and that call writes nothing."""
    g = S.Geometry(2, 4, 2, 64, 1e4)
    w = World(g, 16, spare=0, steps=1)
    seqs = w.rb.answers(1, room=1)
    w.fork([0, 1], 1)
    fits = Q.fork(w.refs, w.table, w.lens, [0] * n, 1, 16) is not None
    assert fits == (n == 40)
    before = [x.clone() for x in (seqs.k8.view(torch.uint8), seqs.k_scale, seqs.refs)]
    seqs.fork([0] * n, 1)
    torch.cuda.synchronize()
    assert P.c2kv_device_error() == (P.C2KV_OK if fits else P.C2KV_EDEVICE)
    if fits:
        w.fork([0] * n, 1)
        w.check(seqs, "all with the first")
    else:
        assert (seqs.n_cached_dev == -1).all() and (seqs.page_table == -1).all()
        assert all(torch.equal(a, b) for a, b in zip(before, (seqs.k8.view(torch.uint8), seqs.k_scale, seqs.refs)))
    w.sc.close()


def test_fork_behind_a_busy_stream():
    """What a fork lets go of stays until its stream has come to it."""
    g = S.Geometry(2, 4, 2, 64, 1e4)
    tables = []
    for late in (False, True):
        w = World(g, 16, spare=60)
        seqs = w.rb.answers(2, room=3)
        parents = torch.tensor([3, 0, -1, 2, 2], dtype=torch.int32, device="cuda")
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        shapes = [(x.shape, x.dtype) for x in (seqs.page_table, seqs.n_cached_dev, seqs.rope_start, parents)]
        if late:
            with torch.cuda.stream(side):
                torch.cuda._sleep(200_000_000)
            seqs.fork(parents, 20, side)
            del parents
            junk = [torch.full(s, -1, dtype=t, device="cuda") for s, t in shapes for _ in range(3)]
        else:
            seqs.fork(parents, 20)
        torch.cuda.synchronize()
        assert P.c2kv_device_error() == P.C2KV_OK
        tables.append((seqs.page_table.clone(), seqs.n_cached_dev.clone(), seqs.rope_start.clone(), seqs.refs.clone()))
        w.sc.close()
    assert all(int((x != -1).sum()) == 0 for x in junk)
    for a, b in zip(*tables):
        assert torch.equal(a, b)


def test_a_larger_chunk_between_capture_and_replay():
    """A captured chunk keeps its workspace when a larger one is asked for."""
    g = S.Geometry(2, 4, 2, 64, 1e4)
    w = World(g, 16, spare=120, steps=120)   # max_keys is the request's rows and 120
    seqs = w.rb.answers(2, room=100)

    def args(t):
        q = _dev(_values(w.rng, (4, t, 4, 64)))
        k, v = (_dev(_values(w.rng, (4, t, 2, 64))) for _ in range(2))
        return q, k, v, torch.zeros_like(q)

    small, large = args(3), args(90)
    seqs.chunk(0, *small)
    torch.cuda.synchronize()
    size = seqs._chunk_ws[-1].numel()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        seqs.chunk(0, *small)
    seqs.chunk(0, *large)
    assert seqs._chunk_ws[-1].numel() > size
    seqs.chunk(0, *small)
    torch.cuda.synchronize()
    want = small[3].clone()
    junk = [torch.full((size,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(3)]
    small[3].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert P.c2kv_device_error() == P.C2KV_OK
    assert all(bool((x == 0x5A).all()) for x in junk)
    assert torch.equal(small[3], want)
    w.sc.close()
