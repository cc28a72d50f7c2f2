"""Attention of a chunk of new tokens over the 8-bit pages against the fp64
oracle (oracle/pages8_oracle.py).

Bars.  Codes and scales: equal (the append is c2kv_pages8_append's).  Output: its
own bf16 rounding, 2^-8 |ref|; the queries are held in fp16, half a step of which
is 2^-11, so a logit is off by at most ds = 2^-11 sum_i |q_i K_ji| / sqrt(d)
(rotation and sums in fp32 add 2^-18 of the same sum), which moves a convex mean
of V by at most 2 ds max|V|; the weights, in fp16 as well, by 2^-11 max|V|, and
what they lose below fp16's normal range, 2^-31 of the largest each, by 2^-31 of
the number of rows.  In the mean square the output is within 1.2 times what a
rounding to bf16 may be off, 2^-8 / sqrt(3) of its own.
"""
import numpy as np
import pytest
import torch

import oracle.pages8_oracle as Q
import compressed_composable_kv_gb300 as P
from compressed_composable_kv_gb300 import synth as S
from test_gpu_pages8 import Pool, _dev, _f64, _geom, _ok, _rope, _rotate, _round_key, _values

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


class Chunk:
    """A pool with sequences of `held` rows and `new` tokens behind them."""

    def __init__(self, g, page, held, new, t_len=None, seed=0, sharp=1.0, kind="normal", start=None, extra_pages=1):
        t_len = max(new) if t_len is None else t_len
        self.g, self.page, self.held, self.new, self.t_len = g, page, held, new, t_len
        total = [max(0, h) + n for h, n in zip(held, new)]
        need = -(-t_len // page)
        pool = self.pool = Pool(g, page, total, seed=seed, extra_pages=max(extra_pages, need))
        rng, b, h, d = pool.rng, len(held), g.n_kv_heads, g.head_dim
        for kv in (0, 1):
            for i, n in enumerate(held):
                if n > 0:
                    x = _f64(_values(rng, (h, n, d), kind))
                    if kind == "wild":   # pages of very different scales, numbers whose products stay in range
                        x = _f64(_values(rng, (h, n, d))) * np.exp2(np.repeat(rng.integers(-9, 3, (h, -(-n // page))), page, 1)[:, :n, None])
                    pool.put(0, i, 0, kv, x)
        pool.upload()
        k_kind = "normal" if kind == "wild" else kind
        self.q = _values(rng, (b, t_len, g.n_q_heads, d))
        self.q = torch.from_numpy(_f64(self.q) * sharp).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
        self.k, self.v = (_values(rng, (b, t_len, h, d), k_kind) for _ in range(2))
        self.pos = (rng.integers(0, 131072 - t_len, b) if start is None else np.asarray(start))[:, None] + np.arange(t_len)
        self.tab = _rope(g, self.pos)
        self.row = _i32(np.arange(b) * t_len)
        self.n = _i32(held)
        self.n_new = None if all(n == t_len for n in new) else _i32(new)
        self.most = max(total)
        self.ws = torch.full((P.c2kv_attend_pages8_chunk_workspace_size(g, b, t_len, self.most),), 0xA5, dtype=torch.uint8,
                             device="cuda")   # of any contents
        self.out = torch.full((b, t_len, g.n_q_heads, d), -7.0, dtype=torch.bfloat16, device="cuda")

    def call(self, **kw):
        a = dict(n_cached=self.n, max_keys=self.most, tab=self.tab, row=self.row, n_new=self.n_new, ws=self.ws, out=self.out,
                 layer=0, flags=0, stream=None)
        a.update(kw)
        for name, bits in (("q", self.q), ("k_new", self.k), ("v_new", self.v)):
            if name not in a:   # no copies while a graph is captured
                a[name] = _dev(bits)
        P.c2kv_attend_pages8_chunk(self.g, a["layer"], *self.pool.args(), a["n_cached"], a["max_keys"], a["q"], a["k_new"], a["v_new"],
                                   a["tab"], a["row"], a["out"], a["ws"], a["n_new"], stream=a["stream"], flags=a["flags"])
        return a["out"]

    def put_new(self, only=None):
        for b, (h, n) in enumerate(zip(self.held, self.new)):
            if h < 0 or n == 0 or (only is not None and b not in only):
                continue
            kr = _round_key(_rotate(self.g, _f64(self.k[b, :n]), self.pos[b, :n]))
            self.pool.put(0, b, h, 0, kr.transpose(1, 0, 2))
            self.pool.put(0, b, h, 1, _f64(self.v[b, :n]).transpose(1, 0, 2))

    def check(self, what="", rows=None, only=None):
        """Codes, and the outputs (of these rows of each sequence, if given)."""
        self.pool.check(what)
        got_all = self.out.float().cpu().numpy().astype(np.float64)
        g, pl = self.g, self.pool
        for b, (h, n) in enumerate(zip(self.held, self.new)):
            live = 0 if h < 0 or (only is not None and b not in only) else n
            assert (got_all[b, live:] == -7.0).all(), f"{what}: sequence {b} written behind its tokens"
            if live == 0:
                continue
            k, v = (Q.held(pl.codes[x][0], pl.scales[x][0], self.page, pl.table[b], h + n) for x in (0, 1))
            q = _rotate(g, _f64(self.q[b, :n]), self.pos[b, :n])
            pick = range(n) if rows is None else sorted({i % n for i in rows})
            sq_err = sq_ref = 0.0
            for i in pick:
                with np.errstate(invalid="ignore"):
                    ref = Q.attend(q[i], k[:, :h + i + 1], v[:, :h + i + 1])
                got = got_all[b, i]
                bad = ~np.isfinite(ref)
                assert np.array_equal(np.isnan(got), bad), f"{what}: sequence {b} token {i}: NaN in other places"
                kk, vv = np.abs(k[:, :h + i + 1]), np.abs(v[:, :h + i + 1])
                group = g.n_q_heads // g.n_kv_heads
                for kvh in range(g.n_kv_heads):
                    heads = slice(kvh * group, (kvh + 1) * group)
                    if bad[heads].any():
                        continue
                    ds = (2.0 ** -11 + 2.0 ** -18) * (np.abs(q[i, heads]) @ kk[kvh].T).max(-1) / np.sqrt(g.head_dim)
                    tol = 2.0 ** -8 * np.abs(ref[heads]) + ((2 * ds + 2.0 ** -11 + 2.0 ** -31 * (h + n)) * vv[kvh].max())[:, None]
                    err = np.abs(got[heads] - ref[heads])
                    assert (err <= tol).all(), f"{what}: sequence {b} token {i} head {kvh}: {err.max():.3e}, {(err / tol).max():.2f} of the bar"
                    sq_err += (err ** 2).sum()
                    sq_ref += (ref[heads] ** 2).sum()
            assert sq_err <= (1.2 * 2.0 ** -8) ** 2 / 3 * sq_ref, f"{what}: sequence {b}: {np.sqrt(sq_err / sq_ref):.2e} in the mean square"


SHAPES = [(128, 1), (128, 2), (128, 4), (128, 5), (128, 8), (64, 1), (64, 2), (64, 4), (64, 5), (64, 8)]


@pytest.mark.parametrize("d,group", SHAPES)
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_chunk(d, group, page):
    """Lengths around pages and tiles, empty places, a sequence without new
    tokens, ragged chunks behind which nothing is written."""
    g = _geom(d, group, 2)
    held = [0, 1, page - 1, page, 127, 128, 129, 400, -1, 300, 255]
    new = [7, 1, 3, 9, 2, 1, 9, 5, 4, 0, 8]
    c = Chunk(g, page, held, new, t_len=9, seed=d + group + page)
    c.call()
    _ok()
    c.put_new()
    c.check(f"d{d} group {group} page {page}")


@pytest.mark.parametrize("d,group", [(128, 4), (128, 5), (64, 8), (64, 1)])
@pytest.mark.parametrize("t_len", [1, 2, 31, 64, 65, 129, 257, 300])
def test_chunk_lengths(d, group, t_len):
    """Chunks of one token to several hundred, on an empty cache and a long one."""
    g = _geom(d, group, 2)
    c = Chunk(g, 32, [0, 700, 1500], [t_len, t_len, max(1, t_len - 1)], t_len=t_len, seed=t_len, sharp=3.0)
    c.call()
    _ok()
    c.put_new()
    c.check(f"d{d} group {group} t {t_len}", rows=[0, 1, 15, 31, 32, 50, 51, 63, 64, 127, 128, 255, 256, t_len - 2, t_len - 1])


def test_long_cache_and_many_sequences():
    """Units shared by many CTAs, and many units to a CTA."""
    g = _geom(128, 4, 2)
    c = Chunk(g, 64, [20000, 3], [70, 70], seed=1)
    c.call()
    _ok()
    c.put_new()
    c.check("long", rows=[0, 31, 32, 69])
    g = _geom(128, 8, 4)
    held = [(37 * i * i) % 900 for i in range(120)]
    new = [1 + i % 40 for i in range(120)]
    c = Chunk(g, 16, held, new, seed=2)
    c.call()
    _ok()
    c.put_new()
    c.check("many", rows=[0, 17, 39])


def test_256_sequences():
    g = _geom(64, 2, 2)
    held = [-1 if i % 11 == 5 else (i * 7) % 100 for i in range(256)]
    c = Chunk(g, 16, held, [i % 4 for i in range(256)], t_len=3, seed=3)
    c.call()
    _ok()
    c.put_new()
    c.check("256 sequences")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
def test_pages_of_very_different_scales(d, page):
    g = _geom(d, 4, 2)
    c = Chunk(g, page, [1000, 333], [150, 150], seed=d + page, kind="wild")
    c.call()
    _ok()
    c.put_new()
    c.check("scales", rows=range(0, 150, 7))


@pytest.mark.parametrize("d", [64, 128])
def test_values_that_are_not_finite(d):
    """A held NaN answers NaN to the tokens that see it, in its columns, and to
    no others; neither do keys and values behind a token."""
    g = _geom(d, 4, 2)
    c = Chunk(g, 32, [100, 100, 0], [150, 20, 40], t_len=150, seed=d)
    c.v[0, 37, 0, 5], c.v[0, 120, 1, d - 1], c.v[2, 20, 0, 0] = 0x7FC0, 0x7F80, 0xFF80   # NaN, inf, -inf
    c.k[1, 7, 1, 3] = 0x7FC0
    c.pool.codes[1][0, c.pool.table[1, 1], 0, 3, 9] = 0x7F   # a held value that every token sees
    c.pool.upload()
    c.call()
    _ok()
    c.put_new()
    c.check("not finite")


def test_queries_that_are_not_finite():
    g = _geom(128, 2, 2)
    c = Chunk(g, 32, [300], [40], seed=5)
    c.q[0, 3, 1, 7], c.q[0, 9, 2, 100] = 0x7F80, 0x7FC0
    c.call()
    _ok()
    out = c.out.float().cpu().numpy()
    bad = np.isnan(out)
    want = np.zeros((40, 4), bool)
    want[3, 1] = want[9, 2] = True
    assert np.array_equal(bad.all(-1)[0], want) and np.array_equal(bad.any(-1)[0], want)


def test_large_and_small_queries():
    """Queries far above and below fp16's range: their scale is their own."""
    g = _geom(128, 1, 2)
    c = Chunk(g, 64, [200], [6], seed=6)
    f = _f64(c.q) * np.array([1e-30, 2.0 ** -20, 1.0, 20.0, 1e-6, 0.0])[None, :, None, None]
    c.q = torch.from_numpy(f).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    c.call()
    _ok()
    c.put_new()
    c.check("sizes of queries")


def test_missing_pages_are_left_out():
    """A page id outside the pool: an error, its rows take no part, the rest does."""
    g = _geom(128, 4, 2)
    c = Chunk(g, 32, [200, 90], [10, 10], seed=7)
    good = c.pool.table.copy()
    c.pool.table[0, 2], c.pool.table[0, 5] = c.pool.n_pages + 5, -3
    c.pool.upload()
    c.call()
    torch.cuda.synchronize()
    assert P.c2kv_device_error() == P.C2KV_EDEVICE
    c.pool.table = good
    c.put_new()
    out = c.out.float().cpu().numpy().astype(np.float64)
    keep = np.ones(210, bool)
    keep[64:96] = keep[160:192] = False
    k, v = (Q.held(c.pool.codes[x][0], c.pool.scales[x][0], 32, good[0], 210) for x in (0, 1))
    q = _rotate(g, _f64(c.q[0, :10]), c.pos[0, :10])
    for i in range(10):
        m = keep[:200 + i + 1]
        ref = Q.attend(q[i], k[:, :201 + i][:, m], v[:, :201 + i][:, m])
        assert np.abs(out[0, i] - ref).max() < 2e-2 * np.abs(v).max()
    c2 = Chunk(g, 32, [40], [3], seed=8)   # nothing left to attend over but the tokens themselves
    c2.pool.table[0, :2] = -1
    c2.pool.upload()
    c2.call()
    torch.cuda.synchronize()
    assert P.c2kv_device_error() == P.C2KV_EDEVICE
    assert (c2.out == 0).all()


def test_bad_lengths_leave_a_sequence_out():
    g = _geom(128, 4, 2)
    for bad in ("long", "new", "less", "row", "table"):
        c = Chunk(g, 32, [100, 60, 30], [8, 8, 8], t_len=8, seed=9)
        n, new, row, most = [100, 60, 30], [8, 8, 8], [0, 8, 16], 108
        if bad == "long":
            n[1] = 101
        elif bad == "new":
            new[1] = 9
        elif bad == "less":
            new[1] = -1
        elif bad == "row":
            row[1] = -1
        else:
            row[1] = 17
        c.call(n_cached=_i32(n), n_new=_i32(new), row=_i32(row), max_keys=most)
        torch.cuda.synchronize()
        assert P.c2kv_device_error() == P.C2KV_EDEVICE, bad
        c.put_new(only=(0, 2))
        c.check(bad, only=(0, 2))


def test_rows_held_already():
    """k_new and v_new None: the same answers over rows that were appended before,
    and nothing is written to the pages."""
    g = _geom(128, 4, 2)
    a = Chunk(g, 32, [100, 0, 77], [33, 20, 1], t_len=33, seed=10)
    want = a.call().clone()
    before = [t.clone() for t in a.pool.args()]
    a.out.fill_(-7.0)
    got = a.call(k_new=None, v_new=None)
    _ok()
    assert torch.equal(got, want)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(before, a.pool.args()))


def test_one_token_is_the_decode_step():
    """t_len 1 answers as c2kv_attend_pages8 does and leaves the same pages."""
    g = _geom(128, 5, 2)
    held = [5, 900, 64, -1, 127]
    a, b = (Chunk(g, 16, held, [1] * 5, seed=11) for _ in range(2))
    a.call()
    b.out.fill_(-7.0)
    ws = torch.zeros(P.c2kv_attend_pages8_workspace_size(g, 5, 901), dtype=torch.uint8, device="cuda")
    P.c2kv_attend_pages8(g, 0, *b.pool.args(), b.n, 901, _dev(b.q)[:, 0].contiguous(), _dev(b.k)[:, 0].contiguous(),
                         _dev(b.v)[:, 0].contiguous(), b.tab, b.row, b.out.view(5, 10, 128), ws)
    _ok()
    a.put_new()
    a.check("chunk")
    b.put_new()
    b.check("decode")


def test_row_at_length():
    """C2KV_DECODE_ROW_AT_LENGTH: rows of the table follow the length."""
    g = _geom(64, 2, 2)
    held, new = [50, 0, 200], [6, 6, 4]
    a = Chunk(g, 16, held, new, t_len=6, seed=12, start=[0, 0, 0])
    first = np.array([7, 1000, 300])
    a.pos = first[:, None] + np.array(held)[:, None] + np.arange(6)
    a.tab = _rope(g, np.arange(1400))
    a.call(row=_i32(first), flags=P.C2KV_DECODE_ROW_AT_LENGTH)
    _ok()
    a.put_new()
    a.check("row at length")


def test_layers_of_a_pool():
    """The layer's own pages; the others' stay as they were."""
    g = _geom(64, 2, 2, layers=3)
    c = Chunk(g, 16, [40], [5], seed=13)
    for x in (0, 1):
        c.pool.codes[x][1], c.pool.scales[x][1] = c.pool.codes[x][0], c.pool.scales[x][0]
    c.pool.upload()
    c.call(layer=1)
    _ok()
    for x in (0, 1):   # the oracle writes layer 0: swap it in for layer 1
        c.pool.codes[x][[0, 1]], c.pool.scales[x][[0, 1]] = c.pool.codes[x][[1, 0]], c.pool.scales[x][[1, 0]]
    before = [x.copy() for x in c.pool.codes]
    c.put_new()
    for x in (0, 1):
        c.pool.codes[x][[0, 1]], c.pool.scales[x][[0, 1]] = c.pool.codes[x][[1, 0]], c.pool.scales[x][[1, 0]]
    c.pool.check("layer 1")
    assert before[0].shape[0] == 3


def test_same_bits_from_every_launch_stream_and_graph():
    g = _geom(128, 4, 2)
    c = Chunk(g, 64, [3000, 200, 900], [90, 17, 64], t_len=90, seed=14)
    want = c.call().clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        c.out.fill_(-7.0)
        side.wait_stream(torch.cuda.current_stream())
        c.call(stream=side)
        side.synchronize()
        assert torch.equal(c.out, want)
    kn, vn, q = _dev(c.k), _dev(c.v), _dev(c.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(k_new=kn, v_new=vn, q=q)
        c.call(k_new=kn, v_new=vn, q=q)
    for _ in range(2):
        c.out.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want)
    _ok()


def test_workspace_is_shared_by_calls_of_other_shapes():
    g = _geom(128, 4, 2)
    a, b = Chunk(g, 64, [2500], [100], seed=15), Chunk(g, 16, [40, 600, 9], [3, 3, 3], seed=16)
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    want = [x.call().clone() for x in (a, b)]
    for _ in range(3):
        for x, w in zip((a, b), want):
            x.call(ws=ws)
            assert torch.equal(x.out, w)
    _ok()


def test_pages_beyond_32_bit_offsets():
    """A pool of more than 4 GB of codes a side, the chunk on its last pages."""
    g = _geom(128, 1, 8)
    page, n_pages = 128, 36000
    k8, v8 = (torch.zeros((1, n_pages, 8, page, 128), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (torch.ones((1, n_pages, 8), device="cuda") for _ in range(2))
    table = _i32([[n_pages - 1, n_pages - 3, n_pages - 2]])
    rng = np.random.default_rng(17)
    t, held = 20, 250
    rows = _values(rng, (8, held, 128))
    code = Q.e4m3_codes(np.clip(_f64(rows) * 64, -448, 448))
    for j, pid in enumerate((n_pages - 1, n_pages - 3)):
        part = torch.from_numpy(code[:, 128 * j:128 * j + 128].copy()).cuda()
        for x in (k8, v8):
            x.view(torch.uint8)[0, pid, :, :part.shape[1]] = part
    ks.fill_(2.0 ** -6)
    vs.fill_(2.0 ** -6)
    q, kn, vn = (_values(rng, (1, t, 8, 128)) for _ in range(3))
    pos = np.arange(t)
    ws = torch.zeros(P.c2kv_attend_pages8_chunk_workspace_size(g, 1, t, 270), dtype=torch.uint8, device="cuda")
    out = torch.zeros((1, t, 8, 128), dtype=torch.bfloat16, device="cuda")
    P.c2kv_attend_pages8_chunk(g, 0, k8, v8, ks, vs, table, _i32([held]), 270, _dev(q), _dev(kn), _dev(vn), _rope(g, pos), _i32([0]), out, ws)
    _ok()
    ids = table[0].long()

    def held_rows(x, s):
        return (x.view(torch.uint8)[0, ids].view(torch.float8_e4m3fn).double() * s[0, ids][..., None, None].double()).transpose(0, 1).reshape(8, -1, 128)[:, :270].cpu().numpy()

    k, v = held_rows(k8, ks), held_rows(v8, vs)
    ref = Q.attend_chunk(_rotate(g, _f64(q[0]), pos), k, v, held)
    err = np.abs(out[0].double().cpu().numpy() - ref)
    assert np.sqrt((err ** 2).sum() / (ref ** 2).sum()) < 1.2 * 2.0 ** -8 / np.sqrt(3)


@pytest.mark.parametrize("d,group", [(128, 4), (64, 8)])
@pytest.mark.parametrize("held,new", [([3000, 700, 90], [40, 9, 70]), ([100] * 6, [3] * 6), ([0, 37], [300, 200])])
def test_a_wait_that_runs_out_ends_the_launch(d, group, held, new):
    """The test hook lets a wait of every other CTA run out: the launch ends, says so,
    and the next one is as before."""
    g = _geom(d, group, 4)
    c = Chunk(g, 32, held, new, seed=21)
    good = c.call().clone()
    _ok()
    for _ in range(2):
        P.c2kv_test_expire_next_waits(1)
        c.call()
        torch.cuda.synchronize()
        P.c2kv_test_expire_next_waits(0)
        assert P.c2kv_device_error() == P.C2KV_ETIMEOUT
        c.out.fill_(-7.0)
        assert torch.equal(c.call(), good)
        _ok()


@pytest.mark.parametrize("t_len,held", [(64, 8000), (200, 30000), (33, 500), (700, 600)])
def test_units_of_both_sizes(t_len, held):
    """Rows of 128 and of 256 to a unit, cut and whole, a lengths' end inside a page."""
    g = _geom(128, 4, 4)
    c = Chunk(g, 128, [held, 0], [t_len, t_len // 2], t_len=t_len, seed=t_len, sharp=2.0)
    c.call()
    _ok()
    c.put_new()
    c.check("units", rows=[0, 31, 32, 63, 64, t_len // 2, t_len - 1])


@pytest.mark.parametrize("group,t_len,held", [
    (4, 8, [(53 * i * i) % 870 if i % 9 != 4 else -1 for i in range(30)]),   # two units to a CTA, left whole; empty places
    (5, 170, [3800, 17, 3500, 129]),                                         # one to a CTA, of 256 rows and of 82
    (5, 170, [5600, 5555, 3]),                                               # the same, cut
    (4, 8, [2500] * 20),                                                     # of 32 rows, cut
])
def test_units_left_whole_and_cut(group, t_len, held):
    g = _geom(64, group, 8)
    new = [0 if h < 0 else t_len - (3 * i) % min(t_len, 8) for i, h in enumerate(held)]
    c = Chunk(g, 64, held, new, t_len=t_len, seed=group + t_len)
    c.call()
    _ok()
    c.put_new()
    c.check("%s %s" % (group, t_len), rows=[0, 1, t_len // 2, t_len - 1])


def test_queries_in_the_output_buffer():
    """out may be q itself."""
    g = _geom(128, 4, 2)
    c = Chunk(g, 32, [900, 40], [50, 50], seed=22)
    want = c.call().clone()
    q = _dev(c.q)
    got = c.call(q=q, out=q)
    _ok()
    assert torch.equal(got, want)
