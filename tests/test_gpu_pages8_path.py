"""The 8-bit paged cache where a program uses it: requests composed in bf16,
their question prefilled, the rows taken over into pages, answer tokens decoded
over them (RequestBatch, DecoderModel), and the answer's log probabilities.
Codes and scales are those of the oracle for the bf16 rows (equal); attention
and log probabilities are held to the bars of test_gpu_pages8.py."""
import numpy as np
import pytest
import torch

import oracle.c2kv_oracle as O
import oracle.pages8_oracle as Q
import compressed_composable_kv_gb300 as P
from compressed_composable_kv_gb300 import synth as S
from gpu_util import Scenario, to_bits, upload
from test_gpu_pages8 import _f64, _rotate, _round_key

pytestmark = pytest.mark.gpu


class Requests:
    """Composed and prefilled requests with their pages filled, and the oracle's pages."""

    def __init__(self, g, page, batch=3, q_len=9, steps=5, seed=0xC2D0):
        self.g, self.page, self.steps = g, page, steps
        specs = [(i, 400 + 300 * i, 100 + 75 * i) for i in range(3)]
        requests = [([i % 3, (i + 1) % 3][: 1 + i % 2], None) for i in range(batch)]
        self.sc = Scenario(g, 4, specs, requests, q_len=q_len, decode_steps=steps)
        self.sc.batch = P.RequestBatch(self.sc.store, g, self.sc.reqs, 4, q_len, steps, page8=page)
        w = S.Workload("pages8", g, 4, batch, q_len, steps, seed=seed)
        self.dev = upload(S.make_step_inputs(w))
        self.rb = rb = self.sc.batch
        rb.compose()
        for l in range(g.n_layers):
            if q_len:
                o = torch.empty_like(self.dev["q_pre"][l])
                rb.prefill(l, self.dev["q_pre"][l], self.dev["kq_pre"][l], self.dev["vq"][l], o)
        rb.fill_pages8()
        rb.reset_decode()
        torch.cuda.synchronize()
        assert P.c2kv_device_error() == P.C2KV_OK
        self.table = rb.page_table.cpu().numpy()
        self.rows = [n + q_len for n in rb.n_slots]
        shape = tuple(rb.k8.shape)
        self.codes = [np.zeros(shape, np.uint8) for _ in range(2)]
        self.scales = [np.ones(shape[:3], np.float32) for _ in range(2)]
        for b, n in enumerate(self.rows):
            for l in range(g.n_layers):
                for kv, cache in ((0, rb.k_caches[b]), (1, rb.v_caches[b])):
                    Q.put(self.codes[kv][l], self.scales[kv][l], page, self.table[b], 0, _f64(to_bits(cache[l, :, :n])))

    def step(self, t, outs, overlap=None):
        for l in range(self.g.n_layers):
            self.rb.decode(l, self.dev["qd_pre"][t, l], self.dev["kd_pre"][t, l], self.dev["vd"][t, l], outs[l],
                           overlap_previous=overlap)
        self.rb.advance()

    def outs(self):
        return [torch.empty_like(self.dev["qd_pre"][0, 0]) for _ in range(self.g.n_layers)]

    def oracle_step(self, t):
        """The oracle's append and answer of step t: [layer][sequence] of (output, its bar)."""
        g, rb, got = self.g, self.rb, []
        for l in range(g.n_layers):
            row = []
            for b, n0 in enumerate(self.rows):
                n, pos = n0 + t, rb.l_tot[b] + rb.q_len + t
                kd, vd, qd = (_f64(to_bits(self.dev[k][t, l, b])) for k in ("kd_pre", "vd", "qd_pre"))
                kr = _round_key(_rotate(g, kd[None], [pos]))[0]
                for kv, x in ((0, kr), (1, vd)):
                    Q.put(self.codes[kv][l], self.scales[kv][l], self.page, self.table[b], n, x[:, None])
                K, V = (Q.held(self.codes[i][l], self.scales[i][l], self.page, self.table[b], n + 1) for i in (0, 1))
                qr = _rotate(g, qd[None], [pos])[0]
                ref = Q.attend(qr, K, V)
                ds = 2.0 ** -14 * np.abs(qr).max() * np.abs(K).sum(-1).max() / np.sqrt(g.head_dim)
                row.append((ref, 2.0 ** -8 * np.abs(ref) + (2 * ds + 2.0 ** -11) * np.abs(V).max()))
            got.append(row)
        return got

    def check_pages(self):
        """Every held row and its scale (the rest of a pool holds anything)."""
        rb = self.rb
        for dev, scale, kv in ((rb.k8, rb.k_scale, 0), (rb.v8, rb.v_scale, 1)):
            codes, scales = dev.view(torch.uint8).cpu().numpy(), scale.cpu().numpy()
            for b, n0 in enumerate(self.rows):
                n = int(rb.n_cached_dev[b])
                for l in range(self.g.n_layers):
                    a = Q.held(codes[l], scales[l], self.page, self.table[b], n)
                    r = Q.held(self.codes[kv][l], self.scales[kv][l], self.page, self.table[b], n)
                    assert (a == r).all(), f"layer {l} sequence {b}: {int((a != r).sum())} held values differ"


def _near(outs, want, t):
    for l, row in enumerate(want):
        for b, (ref, tol) in enumerate(row):
            got = outs[l][b].float().cpu().numpy().astype(np.float64)
            assert (np.abs(got - ref) <= tol).all(), f"step {t} layer {l} sequence {b}"


@pytest.mark.parametrize("d,group,page", [(128, 4, 64), (128, 5, 16), (64, 2, 32), (64, 8, 128)])
def test_answer_over_pages(d, group, page):
    """Every step's output and, at the end, every held row, for two layers."""
    r = Requests(S.Geometry(2, 2 * group, 2, d, 5.0e5), page)
    for t in range(r.steps):
        outs = r.outs()
        r.step(t, outs)
        torch.cuda.synchronize()
        assert P.c2kv_device_error() == P.C2KV_OK
        _near(outs, r.oracle_step(t), t)
    r.check_pages()
    r.sc.close()


def test_captured_steps_replay_with_new_lengths_and_pages():
    """Two graphs of one step each, captured once, share the batch's scratch and
    alternate: every replay appends one row further, and a page table changed
    between replays is followed."""
    r = Requests(S.Geometry(2, 8, 2, 128, 5.0e5), 16, steps=6)
    outs = [r.outs(), r.outs()]
    inp = {k: r.dev[k][0].clone() for k in ("qd_pre", "kd_pre", "vd")}

    def one(o):
        for l in range(r.g.n_layers):
            r.rb.decode(l, inp["qd_pre"][l], inp["kd_pre"][l], inp["vd"][l], o[l])
        r.rb.advance()

    graphs = []
    side = torch.cuda.Stream()
    for o in outs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(gr, stream=side):
            one(o)
        graphs.append(gr)
    torch.cuda.synchronize()
    for t in range(r.steps):
        if t == 3:   # the same rows in other pages: the table is read at every replay
            rb = r.rb
            perm = torch.randperm(rb.page_table.numel(), device="cuda")
            new = [torch.empty_like(x) for x in (rb.k8, rb.v8, rb.k_scale, rb.v_scale)]
            for dst, src in zip(new, (rb.k8, rb.v8, rb.k_scale, rb.v_scale)):
                raw = (dst.view(torch.uint8), src.view(torch.uint8)) if dst.dtype == torch.float8_e4m3fn else (dst, src)
                raw[0][:, perm] = raw[1]
            for dst, src in zip((rb.k8, rb.v8, rb.k_scale, rb.v_scale), new):
                dst.copy_(src)
            rb.page_table.copy_(perm[rb.page_table.long()].to(torch.int32))
            p = perm.cpu().numpy()
            for kv in (0, 1):
                c, s = r.codes[kv].copy(), r.scales[kv].copy()
                r.codes[kv][:, p], r.scales[kv][:, p] = c, s
            r.table = rb.page_table.cpu().numpy()
        for k in inp:
            inp[k].copy_(r.dev[k][t])
        graphs[t & 1].replay()
        torch.cuda.synchronize()
        assert P.c2kv_device_error() == P.C2KV_OK
        _near(outs[t & 1], r.oracle_step(t), t)
    r.check_pages()
    r.sc.close()


def test_overlapped_launches_are_those_of_serial_ones():
    """C2KV_DECODE_OVERLAP_PREVIOUS changes when a launch begins, not a bit of
    what it writes; another stream than the current one does neither."""
    res = []
    for overlap, stream in ((False, None), (None, None), (None, torch.cuda.Stream())):
        r = Requests(S.Geometry(4, 32, 8, 128, 5.0e5), 32, batch=4)
        got = []
        torch.cuda.synchronize()
        for t in range(r.steps):
            outs = r.outs()
            for l in range(r.g.n_layers):
                r.rb.decode(l, r.dev["qd_pre"][t, l], r.dev["kd_pre"][t, l], r.dev["vd"][t, l], outs[l], stream, overlap)
            r.rb.advance(stream)
            got.append(outs)
        torch.cuda.synchronize()
        assert P.c2kv_device_error() == P.C2KV_OK
        res.append(torch.stack([torch.stack(o) for o in got]))
        r.sc.close()
    for out in res[1:]:
        assert torch.equal(out, res[0])


@pytest.mark.parametrize("d,batch", [(128, 1), (128, 4), (64, 2)])
def test_wait_timeout_is_reported_and_the_next_launch_is_right(d, batch):
    """The test hook makes a launch wait ~0.5 ms on a barrier nothing arrives on:
    it reports C2KV_ETIMEOUT, and the same step right after is the oracle's."""
    r = Requests(S.Geometry(1, 8, 2, d, 5.0e5), 64, batch=batch)
    P.c2kv_test_expire_next_waits(1)
    outs = r.outs()
    r.rb.decode(0, r.dev["qd_pre"][0, 0], r.dev["kd_pre"][0, 0], r.dev["vd"][0, 0], outs[0])
    torch.cuda.synchronize()
    assert P.c2kv_device_error() == P.C2KV_ETIMEOUT
    P.c2kv_test_expire_next_waits(0)
    r.step(0, outs)
    torch.cuda.synchronize()
    assert P.c2kv_device_error() == P.C2KV_OK
    _near(outs, r.oracle_step(0), 0)
    r.check_pages()
    r.sc.close()


def test_model_step_and_its_log_probabilities():
    """A decoder step over the pages, the LM head and the answer's log
    probabilities in one captured graph: the pages hold what the step's own k
    and v say, and the log probabilities are those of the step's logits."""
    g, shape = S.Geometry(2, 8, 2, 128, 5.0e5), S.ModelShape(512, 1024, 32000, 1e-5)
    r = Requests(g, 64, batch=3, steps=4)
    dev = lambda x: torch.from_numpy(x.view(np.int16)).cuda().view(torch.bfloat16)   # noqa: E731
    w = S.make_decoder_weights(g, shape, 2, seed=5, lm_head=True)
    w = {"layers": [{k: dev(v) for k, v in l.items()} for l in w["layers"]],
         "final_norm": dev(w["final_norm"]), "lm_head": dev(w["lm_head"])}
    m = P.DecoderModel(g, shape, w, 3, top_k=8)
    tokens = torch.tensor([7, -1, 31999], dtype=torch.int32, device="cuda")
    x0 = dev(S.normal_bf16(np.random.default_rng(3), (3, shape.dim)))

    def step():
        m.decode_step(r.rb)
        m.token_logprobs(tokens)

    side = torch.cuda.Stream()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(gr, stream=side):
        step()
    torch.cuda.synchronize()
    for t in range(2):
        m.x.copy_(x0)
        gr.replay()
        torch.cuda.synchronize()
        assert P.c2kv_device_error() == P.C2KV_OK
        lp, ent, ids, tops = Q.token_logprobs(m.logits.double().cpu().numpy(), tokens.cpu().numpy(), 8)
        assert (m.top_ids.cpu().numpy() == ids).all()
        bar = 2.0 ** -17 + 2.0 ** -21 * float(m.logits.float().abs().max())
        for got, ref in ((m.logprob, lp), (m.entropy, ent), (m.top_logprobs, tops)):
            assert np.abs(got.double().cpu().numpy() - ref).max() <= bar + 2.0 ** -21 * np.abs(ref).max()
        # the last layer's own k and v are still in the model's buffers
        for b, n0 in enumerate(r.rows):
            n, pos = n0 + t, r.rb.l_tot[b] + r.rb.q_len + t
            kr = _round_key(_rotate(g, _f64(to_bits(m.k[b])).reshape(1, 2, 128), [pos]))[0]
            vr = _f64(to_bits(m.v[b])).reshape(2, 128)
            for kv, xx, codes, scale in ((0, kr, r.rb.k8, r.rb.k_scale), (1, vr, r.rb.v8, r.rb.v_scale)):
                Q.put(r.codes[kv][1], r.scales[kv][1], 64, r.table[b], n, xx[:, None])
                pid = r.table[b][n // 64]
                a = Q.e4m3_values(codes[1, pid, :, n % 64].view(torch.uint8).cpu().numpy()) * scale[1, pid].cpu().numpy()[:, None]
                want = Q.e4m3_values(r.codes[kv][1][pid, :, n % 64]) * r.scales[kv][1][pid][:, None]
                assert (a == want).all()
    assert int(r.rb.n_cached_dev[0]) == r.rows[0] + 2
    r.sc.close()


def test_shared_pages_and_calls_at_once():
    """Two sequences read the same pages (a shared prefix, nothing appended) and
    answer alike; two batches decoded at once on two streams, each with its own
    pages and scratch, answer as one after the other."""
    a, b = (Requests(S.Geometry(1, 32, 8, 128, 5.0e5), 32, batch=4, seed=s) for s in (1, 2))
    rb = a.rb
    table = rb.page_table.clone()
    table[1] = table[0]
    n = rb.n_cached_dev.clone()
    n[1] = n[0]
    q = a.dev["qd_pre"][0, 0].clone()
    q[1] = q[0]
    row = rb.rope_row_dev.clone()
    row[1] = row[0]
    out = torch.empty_like(q)
    P.c2kv_attend_pages8(a.g, 0, rb.k8, rb.v8, rb.k_scale, rb.v_scale, table, n, rb.max_keys_decode, q, None, None,
                         rb.rope_table, row, out, rb.workspace8)
    torch.cuda.synchronize()
    assert P.c2kv_device_error() == P.C2KV_OK
    assert torch.equal(out[0], out[1]) and out.isfinite().all()

    def run(streams):
        outs = []
        for r, st in zip((a, b), streams):
            r.rb.reset_decode(st)
        torch.cuda.synchronize()
        for t in range(a.steps):
            for r, st in zip((a, b), streams):
                o = torch.empty_like(r.dev["qd_pre"][t, 0])
                r.rb.decode(0, r.dev["qd_pre"][t, 0], r.dev["kd_pre"][t, 0], r.dev["vd"][t, 0], o, st)
                r.rb.advance(st)
                outs.append(o)
        torch.cuda.synchronize()
        assert P.c2kv_device_error() == P.C2KV_OK
        return torch.stack(outs)

    one = torch.cuda.current_stream()
    serial = run((one, one))
    at_once = run((torch.cuda.Stream(), torch.cuda.Stream()))
    assert torch.equal(serial, at_once)
    a.sc.close()
    b.sc.close()


def test_many_launches_give_the_same_bits():
    """Which CTA finishes last varies; what it merges, and in what order, does not."""
    r = Requests(S.Geometry(1, 32, 8, 128, 5.0e5), 16, batch=4)
    outs = []
    for _ in range(40):
        o = torch.empty_like(r.dev["qd_pre"][0, 0])
        r.rb.decode(0, r.dev["qd_pre"][0, 0], r.dev["kd_pre"][0, 0], r.dev["vd"][0, 0], o)
        outs.append(o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
    x = torch.randn(16, 128256, device="cuda").to(torch.bfloat16)
    got = []
    for _ in range(10):
        lp, ent, tops = (torch.empty(s, device="cuda") for s in ((16,), (16,), (16, 12)))
        ids = torch.empty((16, 12), dtype=torch.int32, device="cuda")
        P.c2kv_token_logprobs(x, torch.arange(16, dtype=torch.int32, device="cuda"), 12, lp, ent, ids, tops)
        got.append(torch.cat([lp, ent, ids.float().flatten(), tops.flatten()]))
    assert all(torch.equal(t, got[0]) for t in got[1:])
    r.sc.close()


@pytest.mark.parametrize("d,page", [(128, 64), (64, 16)])
def test_lengths_are_the_only_state_that_advances(d, page):
    """The lengths moved by c2kv_seq_advance, and put back for a step taken
    again: every key is rotated for the place it goes to."""
    r = Requests(S.Geometry(2, 8, 2, d, 5.0e5), page)
    for t in range(r.steps):
        for again in (True, False):
            outs = r.outs()
            for l in range(r.g.n_layers):
                r.rb.decode(l, r.dev["qd_pre"][t, l], r.dev["kd_pre"][t, l], r.dev["vd"][t, l], outs[l])
            P.c2kv_seq_advance(r.rb.n_cached_dev)
            if again:
                r.rb.n_cached_dev.sub_(1)
        torch.cuda.synchronize()
        assert P.c2kv_device_error() == P.C2KV_OK
        _near(outs, r.oracle_step(t), t)
        r.check_pages()
    want = [b * r.rb.cap + n + r.steps for b, n in enumerate(r.rows)]
    assert r.rb.rope_row_dev.tolist() == want
    r.sc.close()


def test_a_step_captured_before_the_pages_are_filled():
    """A program may capture its decode step before the first request's rows are
    there, on the current stream or one it names; run at once, the same call is
    refused, and a fill that is replayed counts."""
    r = Requests(S.Geometry(2, 8, 2, 128, 5.0e5), 32)
    rb, outs = r.rb, r.outs()
    rb.compose()
    for l in range(2):
        o = torch.empty_like(r.dev["q_pre"][l])
        rb.prefill(l, r.dev["q_pre"][l], r.dev["kq_pre"][l], r.dev["vq"][l], o)
    with pytest.raises(ValueError, match="fill_pages8"):
        rb.decode(0, r.dev["qd_pre"][0, 0], r.dev["kd_pre"][0, 0], r.dev["vd"][0, 0], outs[0])
    side = torch.cuda.Stream()
    step, fill = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(step, stream=side):
        for l, st in ((0, None), (1, side.cuda_stream)):
            rb.decode(l, r.dev["qd_pre"][0, l], r.dev["kd_pre"][0, l], r.dev["vd"][0, l], outs[l], st)
        rb.advance()
    with torch.cuda.graph(fill, stream=side):
        rb.fill_pages8()
        rb.compose_layers(0, 2)   # (captured, not run: the rows stay)
    assert rb.filled == {0, 1}
    rb.fill_pages8()
    step.replay()
    torch.cuda.synchronize()
    assert P.c2kv_device_error() == P.C2KV_OK
    _near(outs, r.oracle_step(0), 0)
    r.check_pages()
    r.sc.close()
