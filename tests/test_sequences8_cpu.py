"""PagedSequences without a GPU: what it keeps, gives back and refuses.  The library's
calls are noted, forks are the oracle's."""
import pytest
import torch

import oracle.pages8_oracle as Q
from compressed_composable_kv_gb300 import synth as S
from test_chunk8_cpu import _fork, noted  # noqa: F401
from test_pages8_cpu import P, _pages  # noqa: F401


def _decode(seqs, layer=0):
    x = torch.zeros((seqs.batch, 4, 64))
    seqs.decode(layer, x, x[:, :2], x[:, :2], x)


def test_decode_keeps_one_workspace(noted, P, monkeypatch):  # noqa: F811
    """Its counters are zeroed once, before the first call (a fill while a graph is captured
    would run at its first replay only), and it serves every number of sequences."""
    rb, calls = noted
    used = []
    monkeypatch.setattr(P.pipeline.B, "c2kv_attend_pages8", lambda g, l, *a: used.append(a[13]))
    rb.fill_pages8()
    seqs = rb.answers(2, room=4)
    made = []
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, **kw: made.append(zeros(*a, **kw)) or made[-1])
    _decode(seqs)
    seqs.fork([0, -1, 1], 1)
    _decode(seqs)
    seqs.fork([2], 1)
    _decode(seqs)
    monkeypatch.undo()
    assert len(used) == 3 and all(w is used[0] for w in used)
    assert not any(w.data_ptr() == x.data_ptr() for x in made for w in used) and int(used[0].sum()) == 0
    for batch in (1, 2, 256):
        assert used[0].numel() >= P.c2kv_attend_pages8_workspace_size(seqs.geom, batch, seqs.max_keys)


def _chunk(seqs, t_len):
    x = torch.zeros((seqs.batch, t_len, 4, 64), dtype=torch.bfloat16)
    seqs.chunk(0, x, x[:, :, :2], x[:, :, :2], x)


def test_chunks_keep_one_workspace(noted, P, monkeypatch):  # noqa: F811
    """Chunks longer from call to call: the scratch grows by steps, and what it has grown out of is let go."""
    rb, calls = noted
    used = []
    monkeypatch.setattr(P.pipeline.B, "c2kv_attend_pages8_chunk", lambda g, l, *a: used.append(a[13].numel()))
    rb.fill_pages8()
    seqs = rb.answers(2, room=4)
    for t_len in range(1, 1200, 7):
        _chunk(seqs, t_len)
        assert used[-1] >= P.c2kv_attend_pages8_chunk_workspace_size(seqs.geom, 4, t_len, seqs.max_keys)
    assert len(seqs._chunk_ws) == 1
    assert len(set(used)) < 8


def test_the_pool_is_refused_while_sequences_live_on_it(noted):  # noqa: F811
    """What would write the batch's own rows over pages that answers share is refused until
    the sequences are released, or gone."""
    rb, calls = noted
    x = torch.zeros((2, 4, 64))

    def decode():
        rb.decode(0, x, x[:, :2], x[:, :2], x)

    rb.fill_pages8()
    decode()
    seqs = rb.answers(2, room=4)
    rb.filled.update({0, 1})   # as a program does that writes pages by calls of its own
    for call in (rb.fill_pages8, lambda: rb.fill_pages8(0, 1), decode, lambda: rb.answers(1)):
        with pytest.raises(ValueError, match="release"):
            call()
    _decode(seqs)
    seqs.release()
    n = len(calls)
    for call in (lambda: _decode(seqs), lambda: _chunk(seqs, 2), lambda: seqs.fork([0], 1), seqs.compact):
        with pytest.raises(ValueError, match="released"):
            call()
    assert len(calls) == n
    rb.fill_pages8()
    decode()
    seqs = rb.answers(1)
    with pytest.raises(ValueError, match="release"):
        rb.fill_pages8()
    del seqs
    rb.fill_pages8()
    decode()


@pytest.fixture
def strict(noted, P, monkeypatch):  # noqa: F811
    """As `noted`, with forks that write nothing where the oracle finds none, and the oracle's compaction."""
    rb, calls = noted
    B = P.pipeline.B

    def fork(g, k8, v8, ks, vs, refs, table, n, parent, room, refs_out, table_out, n_out, ws, stream=None):
        got = Q.fork(refs.tolist(), table.tolist(), n.tolist(), parent.tolist(), room, k8.shape[3])
        calls.append(("fork", got is not None))
        if got is not None:
            for dst, src in zip((refs_out, table_out, n_out), got):
                dst.copy_(torch.tensor(src))

    def compact(g, k8, v8, ks, vs, refs, table, refs_out, table_out, moved_out, ws, stream=None):
        got = Q.compact(refs.tolist(), table.tolist())
        for dst, src in zip((refs_out, table_out, moved_out), got):
            if dst is not None:
                dst.copy_(torch.tensor(src))

    monkeypatch.setattr(B, "c2kv_pages8_fork", fork)
    monkeypatch.setattr(B, "c2kv_pages8_compact", compact)
    rb.fill_pages8()
    return rb.answers(2, room=4), calls


def _state(seqs):
    return [x.tolist() for x in (seqs.page_table, seqs.n_cached_dev, seqs.rope_start, seqs.refs)]


@pytest.mark.parametrize("parents,room", [([0] * 40, 4), ([3, 2, 1, 0], 30), ([1], 300), ([0, 1, 2, 3, 7], 1)])
def test_a_failed_fork_loses_nothing(strict, parents, room):
    """Too few pages, more room than a row of the table has, a parent that is none: all
    places are empty, and restore brings back the sequences as they were."""
    seqs, calls = strict
    seqs.advance(n=torch.tensor([2, 0, 1, 3], dtype=torch.int32))
    before = _state(seqs)
    assert not seqs.restore() and _state(seqs) == before   # nothing has failed
    seqs.fork(parents, room)
    assert calls[-1] == ("fork", False)
    assert seqs.batch == len(parents) and (seqs.n_cached_dev == -1).all() and (seqs.page_table == -1).all()
    assert seqs.restore()
    assert _state(seqs) == before
    seqs.fork([3, -1, 0], 2)   # and they go on
    assert calls[-1] == ("fork", True) and seqs.n_cached_dev.tolist() == [16, -1, 15]
    assert not seqs.restore()
    assert sum(seqs.refs.tolist()) == sum(e >= 0 for row in seqs.page_table.tolist() for e in row)


def test_a_failed_fork_is_found_late(strict):
    """Steps go on with the empty places, forks and a compaction among them, before the
    program reads the error: the sequences are still those of before it."""
    seqs, calls = strict
    seqs.fork([0, -1, 3], 1)
    seqs.compact()
    lengths, starts = seqs.n_cached_dev.tolist(), seqs.rope_start.tolist()
    pages = [sum(e >= 0 for e in row) for row in seqs.page_table.tolist()]
    seqs.fork([0, 2] * 9, 20)
    assert calls[-1] == ("fork", False)
    seqs.advance()
    seqs.fork([1, 0, 2], 4)
    seqs.fork(list(range(30)), 1)   # (more places than ever before)
    seqs.compact()
    seqs.advance(n=3)
    assert seqs.restore()
    assert seqs.n_cached_dev.tolist() == lengths and seqs.rope_start.tolist() == starts
    assert [sum(e >= 0 for e in row) for row in seqs.page_table.tolist()] == pages
    assert sum(seqs.refs.tolist()) == sum(pages)


def test_a_compaction_moves_what_a_failed_fork_left(strict):
    seqs, calls = strict
    seqs.fork([2, 3], 4)
    table = seqs.page_table.tolist()
    seqs.fork([0, 1], 300)
    assert calls[-1] == ("fork", False)
    moved = Q.compact(seqs.refs.tolist(), [])[2]
    assert any(m >= 0 and m != i for i, m in enumerate(moved))
    seqs.compact()
    assert seqs.restore()
    assert seqs.page_table.tolist() == [[moved[e] if e >= 0 else -1 for e in row] for row in table]


def test_sequences_that_were_ended_do_not_come_back(strict):
    seqs, calls = strict
    seqs.fork([-1, -1], 1)
    assert calls[-1] == ("fork", True) and sum(seqs.refs.tolist()) == 0
    assert not seqs.restore() and seqs.n_cached_dev.tolist() == [-1, -1]
    seqs.compact()
    seqs.fork([0], 1)
    assert not seqs.restore()


def test_a_failed_fork_of_tensors_that_the_program_has_set(strict):
    seqs, calls = strict
    seqs.fork([0, 1], 4)
    seqs.rope_start = torch.tensor([7, 9], dtype=torch.int32)
    before = _state(seqs)
    seqs.fork([0, 1, 1], 300)
    assert calls[-1] == ("fork", False) and seqs.restore() and _state(seqs) == before


def test_a_table_of_more_entries_than_can_be_counted(P):  # noqa: F811
    """What all places together may take is counted in 32 bits."""
    for batch_out, max_pages in ((256, 1 << 23), (64, 1 << 25), (255, 8421505)):
        assert _fork(P, pages=_pages(P), batch_out=batch_out, max_pages=max_pages) == P.C2KV_EINVAL
        assert "2^31" in P.c2kv_last_error()


def test_pages_that_are_none_do_not_come_back(strict):
    """A table whose entries are no pages makes a fork fail; it is not taken for sequences."""
    seqs, calls = strict
    seqs.page_table[1, 0] = 1 << 30
    seqs.fork([0, 1], 1)
    assert calls[-1] == ("fork", False) and not seqs.restore()
    seqs.compact()
    assert not seqs.restore() and (seqs.n_cached_dev == -1).all()
