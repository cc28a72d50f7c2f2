"""What PagedSequences keeps between calls, on the GPU: workspaces over forks, captures and
growth.  The oracle's pages and bars are test_gpu_sequences8.py's."""
import pytest
import torch

import compressed_composable_kv_gb300 as P
from compressed_composable_kv_gb300 import synth as S
from test_gpu_pages8 import _dev, _values
from test_gpu_pages8_move import Pages
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


def test_chunks_that_grow_on_several_streams():
    """Longer and longer chunks on two streams by turns, each still to run when the next one
    asks for more scratch: the answers are those of one stream, and of a graph captured on the way."""
    g = S.Geometry(1, 4, 2, 64, 1e4)
    w = World(g, 16, spare=160, steps=700)
    seqs = w.rb.answers(2, room=640)
    sides = [torch.cuda.Stream() for _ in range(2)]
    lens = [3, 40, 90, 200, 330, 640]
    args = []
    for t in lens:
        q = _dev(_values(w.rng, (4, t, 4, 64)))
        k, v = (_dev(_values(w.rng, (4, t, 2, 64))) for _ in range(2))
        args.append((q, k, v, torch.zeros_like(q)))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    for i, a in enumerate(args):
        side, other = sides[i % 2], sides[1 - i % 2]
        side.wait_stream(other)   # chunks of one pool follow one another
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        seqs.chunk(0, *a, stream=side)
        if i == 2:
            torch.cuda.synchronize()
            with torch.cuda.graph(graph):
                seqs.chunk(0, *a)
        with torch.cuda.stream(side):   # takes the place of what was let go
            junk = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in (1 << 20, 1 << 22, 1 << 23)]
            del junk
    torch.cuda.synchronize()
    assert P.c2kv_device_error() == P.C2KV_OK
    assert len(seqs._chunk_ws) <= 2   # the captured one and the last
    got = [a[3].clone() for a in args]
    for a, x in zip(args, got):
        a[3].zero_()
        seqs.chunk(0, *a)
        assert torch.equal(a[3], x)
    args[2][3].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(args[2][3], got[2]) and P.c2kv_device_error() == P.C2KV_OK
    w.sc.close()


def test_answers_on_a_stream_given_by_its_handle():
    """A stream is a torch stream or a handle, as in every other call."""
    g = S.Geometry(1, 4, 2, 64, 1e4)
    w = World(g, 16, spare=20)
    side = torch.cuda.Stream()
    seqs = w.rb.answers(2, room=3, stream=side.cuda_stream)
    w.fork([0, 0, 1, 1], 3)
    side.synchronize()
    w.check(seqs, "answers")
    w.sc.close()


@pytest.mark.parametrize("parents,room", [([0] * 250, 1), ([3, 1, 0, 2], 500), ([0, 9], 1)])
def test_sequences_go_on_behind_a_failed_fork(parents, room):
    """Too few pages, more room than the table has, a parent that is none; found after
    further steps, another fork and a compaction."""
    g = S.Geometry(2, 8, 2, 128, 5.0e5)
    w = World(g, 16, spare=25)
    side = torch.cuda.Stream()
    seqs = w.rb.answers(2, room=10)
    w.fork([0, 0, 1, 1], 10)
    w.decode(seqs, 2, "before")
    side.wait_stream(torch.cuda.current_stream())
    seqs.fork(parents, room, side)
    x = [torch.zeros((len(parents), h, 128), dtype=torch.bfloat16, device="cuda") for h in (8, 2, 8)]
    side.wait_stream(torch.cuda.current_stream())
    seqs.decode(0, x[0], x[1], x[1], x[2], side)
    seqs.advance(side)
    seqs.fork([0, 0, 1], 4, side)
    seqs.compact(side)
    w.compact()
    torch.cuda.synchronize()
    assert P.c2kv_device_error() == P.C2KV_EDEVICE
    assert (seqs.n_cached_dev == -1).all()
    assert seqs.restore(side)
    torch.cuda.synchronize()
    w.check(seqs, "restored")
    w.decode(seqs, 2, "restored")
    seqs.fork([2, -1, 0], 3)
    w.fork([2, -1, 0], 3)
    w.chunk(seqs, [2, 0, 3], "restored")
    w.check(seqs, "at the end")
    assert not seqs.restore()
    w.sc.close()


def test_beams_in_a_graph():
    """A step with its fork of the same number of places, captured: the fork's tensors are the
    next step's, so a program copies them back; replays follow the oracle's pages."""
    g = S.Geometry(1, 4, 2, 64, 1e4)
    w = World(g, 16, spare=60)
    seqs = w.rb.answers(2, room=40)
    w.fork([0, 0, 1, 1], 40)
    seqs.fork([0, 1, 2, 3], 1)
    w.fork([0, 1, 2, 3], 1)
    torch.cuda.synchronize()
    was = seqs.page_table, seqs.n_cached_dev, seqs.rope_start
    parents = torch.tensor([1, 0, 2, 2], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        seqs.fork(parents, 1)
        for a, b in zip(was, (seqs.page_table, seqs.n_cached_dev, seqs.rope_start)):
            a.copy_(b)
    seqs.page_table, seqs.n_cached_dev, seqs.rope_start = was
    for step in range(3):
        graph.replay()
        w.fork([1, 0, 2, 2], 1)
        w.check(seqs, f"step {step}")
    w.decode(seqs, 1, "behind the graph")
    w.check(seqs, "behind the graph")
    w.sc.close()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page,room", [(16, 300), (16, 299), (32, 500)])
def test_a_fork_with_much_room(d, page, room):
    """Room for hundreds of tokens in the smallest pages, from a pool that has them."""
    lens = [0, 1, page - 1, page, page + 1, 2 * page, -1, 200, 133]
    p = Pages(lens, page, 500, d=d, width=50, shared=[0, 0, 0, 0, 1, 1, 0, 0, 1], seed=page + d + room)
    want = p.check_fork([8, 0, 8, -1, 2, 3, 3, 3, 6, 7, 4, 4, -5, 5, 5, 8, 1], room)
    assert want is not None and len(want[3]) == 3   # of sequence 8 for two places, of 4 for one
