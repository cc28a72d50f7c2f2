"""Chunk attention over 8-bit pages, forking and compacting without a GPU: pins
of their oracle, and every refusal of the entry points (made before anything is
enqueued)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.pages8_oracle as Q
from compressed_composable_kv_gb300 import synth as S
from test_pages8_cpu import A, P, _pages  # noqa: F401


def test_oracle_chunk_is_torchs_causal_attention():
    rng = np.random.default_rng(0)
    n, t, h, group, d = 5, 4, 2, 3, 16
    q, k, v = rng.standard_normal((t, h * group, d)), rng.standard_normal((h, n + t, d)), rng.standard_normal((h, n + t, d))
    mask = torch.tril(torch.ones(t, n + t), diagonal=n).bool()
    ref = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), torch.from_numpy(k).repeat_interleave(group, 0),
        torch.from_numpy(v).repeat_interleave(group, 0), attn_mask=mask).transpose(0, 1).numpy()
    assert np.abs(Q.attend_chunk(q, k, v, n) - ref).max() < 1e-12


def test_oracle_fork_by_hand():
    """Sequences of 20 and 32 tokens on pages of 16: 0 splits, 1 ends."""
    table = [[4, 2, -1, 9], [0, 5, -1, 1]]
    refs = [1, 0, 1, 0, 1, 1]
    out, rows, n, copies = Q.fork(refs, table, [20, 32], [0, -1, 0], 13, 16)
    # place 0 keeps 4, 2 and takes page 0 (given back) for tokens 32 and on; place 2 shares 4, copies 2 to page 1
    assert rows == [[4, 2, 0, -1], [-1] * 4, [4, 1, 3, -1]]
    assert n == [20, -1, 20] and copies == [(2, 1, 4)]
    assert out == [1, 1, 1, 1, 2, 0]


def test_oracle_compact_by_hand():
    out, rows, moved, moves = Q.compact([0, 2, 0, 0, 1, 1], [[5, 1, -1], [1, 4, -1]])
    assert moves == [(4, 0), (5, 2)]
    assert out == [1, 2, 1, 0, 0, 0] and moved == [-1, 1, -1, -1, 0, 2] and rows == [[2, 1, -1], [1, 0, -1]]


# ------------------------------------------------------------------ refusals

def _chunk(P, g=S.TINY, pages=None, layer=0, batch=1, t_len=3, table=A, max_pages=4, n=A, new=None, max_keys=8, q=A, k=A,
           v=A, rope=A, rows=8, row=A, out=A, ws=A, ws_bytes=1 << 40, flags=0):
    pg = ctypes.byref(pages) if pages is not None else None
    return P.load_library().c2kv_attend_pages8_chunk(ctypes.byref(P.as_geometry(g)), pg, layer, batch, t_len, table,
                                                     max_pages, n, new, max_keys, q, k, v, rope, rows, row, out, ws,
                                                     ws_bytes, flags, None)


def _fork(P, g=S.TINY, pages=None, batch=1, table=A, max_pages=4, n=A, batch_out=2, parent=A, room=1, refs=A, refs_out=A,
          table_out=A, n_out=A, ws=A, ws_bytes=1 << 40):
    pg = ctypes.byref(pages) if pages is not None else None
    return P.load_library().c2kv_pages8_fork(ctypes.byref(P.as_geometry(g)), pg, batch, table, max_pages, n, batch_out,
                                             parent, room, refs, refs_out, table_out, n_out, ws, ws_bytes, None)


def _compact(P, g=S.TINY, pages=None, batch=1, table=A, max_pages=4, refs=A, refs_out=A, table_out=A, moved=None, ws=A,
             ws_bytes=1 << 40):
    pg = ctypes.byref(pages) if pages is not None else None
    return P.load_library().c2kv_pages8_compact(ctypes.byref(P.as_geometry(g)), pg, batch, table, max_pages, refs,
                                                refs_out, table_out, moved, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [_chunk, _fork, _compact])
@pytest.mark.parametrize("bad", [
    dict(pages=None), dict(pages=dict(page=8)), dict(pages=dict(page=48)), dict(pages=dict(n_pages=0)),
    dict(pages=dict(n_pages=(1 << 31) - 1, page=128)), dict(pages=dict(base=4096 + 8)), dict(pages=dict(base=0)),
    dict(batch=0), dict(batch=257), dict(table=None), dict(max_pages=0), dict(max_pages=1 << 28), dict(ws=None),
    dict(ws=A + 4), dict(ws_bytes=8), dict(g=S.Geometry(1, 6, 2, 64, 1e4)), dict(g=S.Geometry(1, 4, 2, 96, 1e4)),
])
def test_refusals(P, call, bad):  # noqa: F811
    bad = dict(bad)
    pages = bad.pop("pages", {})
    assert call(P, pages=None if pages is None else _pages(P, **pages), **bad) == P.C2KV_EINVAL
    assert P.c2kv_last_error()


def test_refusals_of_the_chunk(P):  # noqa: F811
    pg = _pages(P)
    for bad in (dict(layer=-1), dict(layer=1), dict(n=None), dict(rope=None), dict(row=None), dict(rows=0), dict(q=None),
                dict(out=None), dict(k=None), dict(v=None), dict(k=A + 2), dict(v=A + 8), dict(rope=A + 4), dict(q=A + 2),
                dict(out=A + 8), dict(max_keys=0), dict(max_keys=65), dict(flags=1), dict(flags=2), dict(flags=8),
                dict(t_len=0), dict(t_len=-3)):
        assert _chunk(P, pages=pg, **bad) == P.C2KV_EINVAL, bad
    assert _chunk(P, pages=pg, t_len=65) == P.C2KV_ECAPACITY
    many = S.Geometry(1, 256, 256, 64, 1e4)
    assert _chunk(P, g=many, pages=pg, batch=256) == P.C2KV_EINVAL


def test_refusals_of_fork_and_compact(P):  # noqa: F811
    pg = _pages(P)
    for bad in (dict(n=None), dict(parent=None), dict(room=-1), dict(room=1 << 29), dict(batch_out=0), dict(batch_out=257),
                dict(refs=None), dict(refs_out=None), dict(table_out=None), dict(n_out=None)):
        assert _fork(P, pages=pg, **bad) == P.C2KV_EINVAL, bad
    for bad in (dict(refs=None), dict(refs_out=None), dict(table_out=None)):
        assert _compact(P, pages=pg, **bad) == P.C2KV_EINVAL, bad


def test_workspace_sizes(P):  # noqa: F811
    g = S.LLAMA31_8B
    small, large = (P.c2kv_attend_pages8_chunk_workspace_size(g, 4, t, 40000) for t in (4, 512))
    assert 0 < small <= large
    for args in ((0, 4, 10), (257, 4, 10), (1, 0, 10), (1, 4, 0)):
        assert P.c2kv_attend_pages8_chunk_workspace_size(g, *args) == 0
    assert P.c2kv_attend_pages8_chunk_workspace_size(S.Geometry(1, 6, 2, 64, 1e4), 1, 1, 10) == 0
    assert P.c2kv_pages8_plan_workspace_size(1000, 7, 30) >= 4 * (4 * 1000 + 7 * 30)
    for args in ((0, 7, 30), (10, 0, 30), (10, 257, 30), (10, 7, 0)):
        assert P.c2kv_pages8_plan_workspace_size(*args) == 0


def test_binding_checks_shapes_and_types(P):  # noqa: F811
    g = S.TINY
    e4 = torch.float8_e4m3fn
    k8 = torch.zeros((1, 4, 2, 16, 64), dtype=torch.uint8).view(e4)
    sc = torch.ones((1, 4, 2))
    table, two = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    kn, q = torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16), torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16)
    ws, four = torch.zeros(1 << 20, dtype=torch.uint8), torch.zeros(4, dtype=torch.int32)
    pool = dict(k8=k8, v8=k8, k_scale=sc, v_scale=sc, page_table=table)
    chunk = dict(pool, layer=0, n_cached_dev=two, max_keys=10, q=q, k_new=kn, v_new=kn, rope_table=torch.zeros((8, 32, 4)),
                 rope_row_dev=two, out=q, workspace=ws, n_new_dev=two)
    fork = dict(pool, refs=four, n_cached_dev=two, parent_dev=two, room=1, refs_out=four, page_table_out=table,
                n_cached_out=two, workspace=ws)
    compact = dict(pool, refs=four, refs_out=four, page_table_out=table, moved_out=four, workspace=ws)
    for call, good, bads in (
            (P.c2kv_attend_pages8_chunk, chunk, [("q", q[0]), ("q", q.float()), ("k_new", kn[:, :2]), ("out", q[:, :, :2]),
                                                 ("n_new_dev", two.long()), ("rope_row_dev", two[:1]), ("page_table", table[:1]),
                                                 ("q", torch.zeros((2, 4, 3, 64), dtype=torch.bfloat16).transpose(1, 2))]),
            (P.c2kv_pages8_fork, fork, [("refs", four[:3]), ("refs", four.long()), ("parent_dev", table), ("page_table_out", table[:, :3]),
                                        ("page_table_out", table[:1]), ("n_cached_out", two[:1]), ("n_cached_dev", four)]),
            (P.c2kv_pages8_compact, compact, [("refs_out", four[:2]), ("moved_out", two), ("page_table_out", table[:1]),
                                              ("page_table", four)])):
        for name, t in bads + [("k8", k8.view(torch.uint8)), ("v_scale", sc.double()), ("workspace", table.t())]:
            with pytest.raises(ValueError):
                call(g, **dict(good, **{name: t}))
        with pytest.raises(ValueError, match="CUDA"):   # host tensors
            call(g, **good)


# ------------------------------------------------------------------ sequences on shared pages

@pytest.fixture
def noted(P, monkeypatch):  # noqa: F811
    """A paged RequestBatch of two layers on the CPU: its calls of the library are
    noted, a fork done by the oracle."""
    B = P.pipeline.B
    calls = []
    monkeypatch.setattr(B, "c2kv_store_lookup", lambda store, d: (40, 10, 0))
    monkeypatch.setattr(B, "c2kv_workspace_init", lambda ws: None)
    monkeypatch.setattr(B, "c2kv_pages8_fill", lambda *a: None)

    def fork(g, k8, v8, ks, vs, refs, table, n, parent, room, refs_out, table_out, n_out, ws, stream=None):
        got = Q.fork(refs.tolist(), table.tolist(), n.tolist(), parent.tolist(), room, k8.shape[3])
        assert ws.numel() >= P.c2kv_pages8_plan_workspace_size(refs.numel(), max(len(parent), len(n)), table.shape[1])
        for dst, src in zip((refs_out, table_out, n_out), got):
            dst.copy_(torch.tensor(src))
        calls.append(("fork", parent.tolist(), room))

    monkeypatch.setattr(B, "c2kv_pages8_fork", fork)
    monkeypatch.setattr(B, "c2kv_pages8_compact", lambda *a: calls.append(("compact",)))
    monkeypatch.setattr(B, "c2kv_attend_pages8_chunk", lambda g, l, *a: calls.append(("chunk", l, a[-1], a[12].numel())))
    monkeypatch.setattr(B, "c2kv_attend_pages8",
                        lambda g, l, *a: calls.append(("decode", l, bool(a[-1] & B.C2KV_DECODE_OVERLAP_PREVIOUS))))
    rb = P.RequestBatch(None, S.Geometry(2, 4, 2, 64, 1e4), [P.RequestSpec([0]), P.RequestSpec([1])], 4, 3, 20, device="cpu",
                        page8=16, spare_pages=5)
    return rb, calls


def test_answers_share_the_composed_rows(noted):
    rb, calls = noted
    with pytest.raises(ValueError, match="fill_pages8"):
        rb.answers(2)
    rb.fill_pages8()
    with pytest.raises(ValueError):
        rb.answers(0)
    seqs = rb.answers(2, room=4)   # 13 rows of 16 each: one page, which the second answer copies
    assert seqs.page_table.tolist() == [[0, 1, -1], [2, 4, -1], [3, 5, -1], [6, 7, -1]]
    assert seqs.n_cached_dev.tolist() == [13] * 4 and seqs.batch == 4
    assert seqs.rope_start.tolist() == [0, 0, rb.cap, rb.cap]
    assert calls == [("fork", [0, 0, 1, 1], 4)]
    seqs.advance()
    seqs.advance(n=torch.tensor([3, 0, 1, 2], dtype=torch.int32))
    assert seqs.n_cached_dev.tolist() == [17, 14, 15, 16]
    seqs.fork([3, -1, 0], 2)
    assert seqs.n_cached_dev.tolist() == [16, -1, 17] and seqs.rope_start.tolist()[::2] == [rb.cap, 0]
    seqs.advance(n=2)
    assert seqs.n_cached_dev.tolist() == [18, -1, 19]
    assert sum(seqs.refs.tolist()) == sum(e >= 0 for row in seqs.page_table.tolist() for e in row)


def test_what_may_overlap_among_sequences(noted):
    """A decode behind a call that wrote pages or lengths waits for it."""
    rb, calls = noted
    rb.fill_pages8()
    seqs = rb.answers(2, room=4)
    calls.clear()
    x = torch.zeros((4, 4, 64))

    def decode(l, **kw):
        seqs.decode(l, x, x[:, :2], x[:, :2], x, **kw)

    decode(1)
    decode(1)
    decode(0)
    seqs.advance()
    decode(1)
    seqs.chunk(0, x[:, None], x[:, None, :2], x[:, None, :2], x[:, None])
    decode(1)
    seqs.compact()
    decode(1, overlap_previous=True)
    assert [c for c in calls if c[0] == "decode"] == [("decode", 1, False), ("decode", 1, True), ("decode", 0, False),
                                                      ("decode", 1, False), ("decode", 1, False), ("decode", 1, True)]
    chunk = [c for c in calls if c[0] == "chunk"][0]
    assert chunk[1] == 0 and chunk[2] == 4 and chunk[3] > 0


def test_request_batch_refuses_spare_pages_without_pages(P):  # noqa: F811
    for kw in (dict(spare_pages=3), dict(page8=16, spare_pages=-1)):
        with pytest.raises(ValueError, match="spare_pages"):
            P.RequestBatch(None, S.TINY, [], 4, 0, 1, **kw)
