"""What PagedSequences keeps between calls, on the GPU: workspaces over forks, captures and
growth.  The oracle's pages and bars are test_gpu_sequences8.py's."""
import pytest
import torch

import compressed_composable_kv_gb300 as P
from compressed_composable_kv_gb300 import synth as S
from test_gpu_pages8 import _dev, _values
from test_gpu_sequences8 import World

pytestmark = pytest.mark.gpu


def test_first_decode_behind_a_fork_is_captured():
    """A step captured before any other has run with this number of sequences, then the
    same step without the graph, before its first replay."""
    g = S.Geometry(2, 8, 2, 128, 5.0e5)
    w = World(g, 16, spare=90)
    junk = [torch.full((1 << 22,), 0x5A, dtype=torch.uint8, device="cuda") for _ in range(4)]
    del junk   # what is allocated from here on holds anything
    seqs = w.rb.answers(1, room=40)
    w.fork([0, 1], 40)
    w.decode(seqs, 1, "two sequences")
    seqs.fork([0, 0, 1, 1, 1], 40)
    w.fork([0, 0, 1, 1, 1], 40)
    q = _dev(_values(w.rng, (5, 8, 128)))
    k, v = (_dev(_values(w.rng, (5, 2, 128))) for _ in range(2))
    o = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        seqs.decode(0, q, k, v, o)
    w.decode(seqs, 2, "without the graph")
    w.check(seqs, "without the graph")
    seqs.decode(0, q, k, v, o)
    torch.cuda.synchronize()
    want = o.clone()
    o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and P.c2kv_device_error() == P.C2KV_OK
    w.sc.close()
