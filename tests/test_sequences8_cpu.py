"""PagedSequences without a GPU: what it keeps, gives back and refuses.  The library's
calls are noted, forks are the oracle's."""
import pytest
import torch

import oracle.pages8_oracle as Q
from compressed_composable_kv_gb300 import synth as S
from test_chunk8_cpu import noted  # noqa: F401
from test_pages8_cpu import P  # noqa: F401


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
