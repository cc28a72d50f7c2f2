"""The 8-bit paged cache and the token log probabilities without a GPU: pins
of their oracle against torch's own conversions and softmax, and every
refusal of the entry points (made before anything is enqueued)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.pages8_oracle as Q
from compressed_composable_kv_gb300 import build
from compressed_composable_kv_gb300 import synth as S


@pytest.fixture(scope="module")
def P():
    build.build_library()
    import compressed_composable_kv_gb300 as pkg
    pkg.load_library()
    return pkg


def test_oracle_codes_are_torchs():
    """Every code's value, and rounding at, just below and just above every
    midpoint between neighbouring codes."""
    codes = torch.arange(256, dtype=torch.uint8)
    vals = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(vals, Q.E4M3, equal_nan=True)
    pos = Q._POS
    mid = (pos[1:] + pos[:-1]) / 2
    x = np.concatenate([pos, mid, np.nextafter(mid.astype(np.float32), np.float32(0)).astype(np.float64),
                        np.nextafter(mid.astype(np.float32), np.float32(1e9)).astype(np.float64)])
    x = np.concatenate([x, -x, [np.nan]])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(Q.e4m3_codes(x), want)


def test_oracle_scale_is_the_smallest_that_holds_the_rows():
    for a in (448.0, 448.0001, 449.0, 224.0, 224.5, 1.0, 2.0 ** -100, 3e38):
        e = Q.scale_exponent(np.array([0.0, -a]))
        assert a <= 448.0 * 2.0 ** e and a > 448.0 * 2.0 ** (e - 1)
    assert Q.scale_exponent(np.zeros(3)) == Q.MIN_EXPONENT
    assert Q.scale_exponent(np.array([np.inf, np.nan, 1.0])) == -8


def test_oracle_logprobs_are_torchs():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 300)) * 3
    x[2, ::3] = -np.inf
    lp, ent, ids, tops = Q.token_logprobs(x, [0, 299, 1, -1, 7], 4)
    ref = torch.log_softmax(torch.from_numpy(x), -1)
    assert np.allclose(lp, [ref[0, 0], ref[1, 299], ref[2, 1], 0.0, ref[4, 7]], atol=1e-12)
    assert np.allclose(ent, torch.special.entr(ref.exp()).sum(-1).numpy(), atol=1e-12)
    v, i = torch.sort(torch.from_numpy(x), dim=-1, descending=True, stable=True)
    assert np.array_equal(ids, i[:, :4].numpy())
    assert np.allclose(tops, ref.gather(1, i[:, :4]).numpy(), atol=1e-12)


# ------------------------------------------------------------------ refusals

def _pages(P, page=16, n_pages=4, base=4096):
    return P.c2kv_pages8(base, base, base, base, n_pages, page)


A = 4096   # a made-up aligned device address: no call below gets as far as using it


def _append(P, g=S.TINY, pages=None, layer=0, batch=1, t_len=1, table=A, max_pages=4, n=A, new=None, k=A, v=A, rope=A,
            rows=8, row=A):
    pg = ctypes.byref(pages) if pages is not None else None
    return P.load_library().c2kv_pages8_append(ctypes.byref(P.as_geometry(g)), pg, layer, batch, t_len, table, max_pages,
                                               n, new, k, v, rope, rows, row, None)


def _attend(P, g=S.TINY, pages=None, layer=0, batch=1, table=A, max_pages=4, n=A, max_keys=8, q=A, k=A, v=A, rope=A,
            rows=8, row=A, out=A, ws=A, ws_bytes=1 << 30, flags=0):
    pg = ctypes.byref(pages) if pages is not None else None
    return P.load_library().c2kv_attend_pages8(ctypes.byref(P.as_geometry(g)), pg, layer, batch, table, max_pages, n,
                                               max_keys, q, k, v, rope, rows, row, out, ws, ws_bytes, flags, None)


@pytest.mark.parametrize("call", [_append, _attend])
@pytest.mark.parametrize("bad", [
    dict(pages=None), dict(pages=dict(page=8)), dict(pages=dict(page=48)), dict(pages=dict(page=256)),
    dict(pages=dict(n_pages=0)), dict(pages=dict(n_pages=(1 << 31) - 1, page=128)), dict(pages=dict(base=4096 + 8)),
    dict(pages=dict(base=0)), dict(layer=-1), dict(layer=1), dict(batch=0), dict(batch=257), dict(table=None),
    dict(max_pages=0), dict(max_pages=1 << 28), dict(n=None), dict(rope=None), dict(row=None), dict(rows=0),
    dict(k=A + 2), dict(v=A + 8), dict(rope=A + 4), dict(g=S.Geometry(1, 6, 2, 64, 1e4)),
    dict(g=S.Geometry(1, 4, 2, 96, 1e4)),
])
def test_refusals_over_pages(P, call, bad):
    bad = dict(bad)
    pages = bad.pop("pages", {})
    assert call(P, pages=None if pages is None else _pages(P, **pages), **bad) == P.C2KV_EINVAL
    assert P.c2kv_last_error()


def test_refusals_of_append_and_attend_alone(P):
    pg = _pages(P)
    assert _append(P, pages=pg, t_len=0) == P.C2KV_EINVAL
    assert _append(P, pages=pg, k=None) == P.C2KV_EINVAL
    assert _append(P, pages=pg, t_len=65) == P.C2KV_ECAPACITY      # 4 pages of 16
    many = S.Geometry(1, 256, 256, 64, 1e4)
    assert _append(P, g=many, pages=pg, batch=256) == P.C2KV_EINVAL     # 65536 heads of sequences
    for bad in (dict(q=None), dict(out=None), dict(ws=None), dict(ws=A + 4), dict(k=None), dict(v=None), dict(q=A + 2),
                dict(max_keys=0), dict(max_keys=65), dict(flags=2), dict(ws_bytes=64)):
        assert _attend(P, pages=pg, **bad) == P.C2KV_EINVAL, bad


def test_refusals_of_fill(P):
    lib = P.load_library()
    g = S.Geometry(2, 4, 2, 64, 1e4)

    def call(begin=0, end=2, batch=1, caches=(A,), cap=64, rows=(10,), max_pages=4, pages=None):
        arr = (ctypes.c_void_p * max(1, len(caches)))(*caches)
        pages = _pages(P) if pages is None else pages
        return lib.c2kv_pages8_fill(ctypes.byref(P.as_geometry(g)), ctypes.byref(pages), begin, end, batch, arr, arr, cap,
                                    (ctypes.c_int32 * len(rows))(*rows), A, max_pages, None)

    for bad in (dict(begin=-1), dict(begin=1, end=1), dict(end=3), dict(batch=0), dict(batch=17, caches=(A,) * 17, rows=(1,) * 17),
                dict(caches=(0,)), dict(caches=(A + 2,)), dict(cap=0), dict(rows=(-1,))):
        assert call(**bad) == P.C2KV_EINVAL, bad
    assert call(rows=(65,)) == P.C2KV_ECAPACITY
    assert call(cap=200, rows=(65,)) == P.C2KV_ECAPACITY
    assert call(rows=(0,)) == P.C2KV_OK     # nothing to do


def test_refusals_of_logprobs(P):
    lib = P.load_library()

    def call(x=A, dtype=0, rows=2, vocab=10, stride=10, tokens=A, k=3, lp=A, ent=A, ids=A, tops=A):
        return lib.c2kv_token_logprobs(x, dtype, rows, vocab, stride, tokens, k, lp, ent, ids, tops, None)

    for bad in (dict(x=None), dict(x=A + 1), dict(dtype=2), dict(dtype=1, x=A + 2), dict(rows=-1), dict(vocab=0),
                dict(vocab=(1 << 30) + 1, stride=1 << 31), dict(stride=9), dict(k=-1), dict(k=11), dict(k=65, vocab=100, stride=100),
                dict(tokens=None), dict(lp=None), dict(ids=None), dict(tops=None)):
        assert call(**bad) == P.C2KV_EINVAL, bad
    assert call(rows=0) == P.C2KV_OK


def test_workspace_size(P):
    g = S.LLAMA31_8B
    assert P.c2kv_attend_pages8_workspace_size(g, 4, 32769) > 0
    for args in ((0, 10), (257, 10), (1, 0)):
        assert P.c2kv_attend_pages8_workspace_size(g, *args) == 0
    assert P.c2kv_attend_pages8_workspace_size(S.Geometry(1, 6, 2, 64, 1e4), 1, 10) == 0


def test_binding_checks_shapes_and_types(P):
    g = S.TINY
    e4 = torch.float8_e4m3fn
    k8 = torch.zeros((1, 4, 2, 16, 64), dtype=torch.uint8).view(e4)
    sc = torch.ones((1, 4, 2))
    table, one = torch.zeros((1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    kn = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16)
    rope = torch.zeros((8, 32, 4))
    good = dict(k8=k8, v8=k8, k_scale=sc, v_scale=sc, page_table=table, n_cached_dev=one, k_new=kn, v_new=kn)
    for name, t in (("k8", k8.view(torch.uint8)), ("v8", k8[:, :3]), ("k_scale", sc.double()), ("v_scale", sc[:, :, :1]),
                    ("page_table", table.long()), ("page_table", torch.zeros((2, 4), dtype=torch.int32)),
                    ("k8", k8[0]), ("k8", k8.transpose(1, 2))):
        with pytest.raises(ValueError):
            P.c2kv_pages8_append(g, 0, **dict(good, **{name: t}), rope_table=rope, rope_row_dev=one)
    x = torch.zeros((2, 10))
    with pytest.raises(ValueError, match="side by side"):
        P.c2kv_token_logprobs(x.t(), None, 0, None, None)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        P.c2kv_token_logprobs(x.half(), None, 0, None, None)


def test_request_batch_refuses_other_page_sizes(P):
    for page8 in (0, 8, 48, 256):
        with pytest.raises(ValueError, match="page8"):
            P.RequestBatch(None, S.TINY, [], 4, 0, 1, page8=page8)


@pytest.fixture
def paged_batch(P, monkeypatch):
    """A paged RequestBatch of two layers on the CPU: its calls of the library
    are noted, not made."""
    B = P.pipeline.B
    calls = []
    monkeypatch.setattr(B, "c2kv_store_lookup", lambda store, d: (40, 10, 0))
    monkeypatch.setattr(B, "c2kv_workspace_init", lambda ws: None)
    monkeypatch.setattr(B, "c2kv_compose_layers", lambda *a: (10, 40))
    monkeypatch.setattr(B, "c2kv_attend_prefill", lambda *a: None)
    monkeypatch.setattr(B, "c2kv_pages8_fill", lambda g, l0, l1, *a: calls.append(("fill", l0, l1)))
    monkeypatch.setattr(B, "c2kv_attend_pages8",
                        lambda g, l, *a: calls.append(("attend", l, bool(a[-1] & B.C2KV_DECODE_OVERLAP_PREVIOUS))))
    g = S.Geometry(2, 4, 2, 64, 1e4)
    rb = P.RequestBatch(None, g, [P.RequestSpec([0]), P.RequestSpec([1])], 4, 3, 5, device="cpu", page8=16)
    x = torch.zeros((2, 4, 64))

    def decode(layer, **kw):
        rb.decode(layer, x, x[:, :2], x[:, :2], x, **kw)

    return rb, decode, calls


def test_pages_that_do_not_hold_the_rows_are_refused(paged_batch):
    """Before fill_pages8, and after rows were composed or prefilled anew: of
    the layers concerned alone."""
    rb, decode, calls = paged_batch

    def refused():
        bad = []
        for l in (0, 1):
            calls.clear()
            try:
                decode(l)
            except ValueError as e:
                assert f"layer {l}" in str(e) and "fill_pages8" in str(e) and not calls
                bad.append(l)
        return bad

    rb.compose()
    assert refused() == [0, 1]
    rb.fill_pages8(0, 1)
    assert refused() == [1]
    rb.fill_pages8()
    assert refused() == []
    rb.prefill(1, None, None, None, None)
    assert refused() == [1]
    rb.fill_pages8(1, 2)
    rb.compose_layers(0, 1)
    assert refused() == [0]
    rb.filled.add(0)     # by a program that wrote the pages itself
    assert refused() == []


def test_a_step_behind_a_fill_does_not_overlap_it(paged_batch):
    """C2KV_DECODE_OVERLAP_PREVIOUS reads the layer's pages before the kernel
    before is done, so the first step behind a fill goes without; a caller that
    asks for either gets it."""
    rb, decode, calls = paged_batch
    rb.compose()
    for l in (0, 1):
        rb.fill_pages8(l, l + 1)
        decode(l)
    decode(1)
    decode(0)
    decode(1, overlap_previous=False)
    decode(0, overlap_previous=True)
    rb.fill_pages8()
    decode(0)
    decode(1)
    want = [("fill", 0, 1), ("attend", 0, False), ("fill", 1, 2), ("attend", 1, False), ("attend", 1, True),
            ("attend", 0, False), ("attend", 1, False), ("attend", 0, True), ("fill", 0, 2), ("attend", 0, False),
            ("attend", 1, True)]
    assert calls == want


def test_log_probabilities_need_an_lm_head(P, monkeypatch):
    monkeypatch.setattr(P.pipeline.B, "c2kv_workspace_init", lambda ws: None)
    m = P.DecoderModel(S.TINY, S.ModelShape(64, 128, 32, 1e-5), {"layers": []}, 2, device="cpu", top_k=3)
    with pytest.raises(ValueError, match="lm_head"):
        m.token_logprobs(torch.zeros(2, dtype=torch.int32))


@pytest.fixture
def fake_build(tmp_path, monkeypatch):
    """A build into an empty folder whose compilers only make their outputs;
    `gxx` says what becomes of g++: its return code, or None: there is none."""
    state = dict(gxx=0, ran=[])
    for name, file in (("LIB", "libc2kv.so"), ("MARSHAL", "_marshal.so")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")

    def run(cmd, **kw):
        state["ran"].append(cmd[0])
        if cmd[0] == "g++" and state["gxx"] is None:
            raise FileNotFoundError("g++")
        code = state["gxx"] if cmd[0] == "g++" else 0
        if code == 0:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return build.subprocess.CompletedProcess(cmd, code, "", "no such header")

    monkeypatch.setattr(build.subprocess, "run", run)
    return state


@pytest.mark.parametrize("gxx", [1, None])
def test_the_library_is_built_where_the_marshalling_module_cannot_be(fake_build, gxx, capsys):
    import os
    fake_build["gxx"] = gxx
    open(build.MARSHAL, "w").close()    # of an older source: not to be loaded
    os.utime(build.MARSHAL, (0, 0))
    assert build.build_library() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.MARSHAL) and "_marshal.so" in capsys.readouterr().err
    fake_build.update(gxx=0, ran=[])
    build.build_library()
    assert os.path.exists(build.MARSHAL) and "nvcc" not in fake_build["ran"]
    fake_build["ran"] = []
    build.build_library()
    assert fake_build["ran"] == []


def test_the_marshalling_module_belongs_to_one_torch(fake_build, monkeypatch, tmp_path):
    """Built anew for another torch, and not loaded before it is."""
    from compressed_composable_kv_gb300 import binding
    build.build_library()
    assert build.up_to_date()
    other = tmp_path / "site" / "torch"
    other.mkdir(parents=True)
    (other / "version.py").write_text("__version__ = '0.0'\n")
    monkeypatch.setattr(build, "_torch_dir", lambda: str(other))
    assert not build.up_to_date()
    monkeypatch.setattr(binding, "MARSHAL", build.MARSHAL)
    monkeypatch.setattr(binding, "load_library", lambda: None)
    with pytest.raises(ImportError, match="another torch"):
        binding._load_marshal()
    fake_build["ran"] = []
    build.build_library()
    assert build.up_to_date() and fake_build["ran"] == ["g++", "g++"]


def test_a_marshalling_module_build_cut_short_is_not_taken_for_done(fake_build, monkeypatch):
    build.build_library()
    assert build.marshal_fits_torch()
    real = build.os.replace

    def cut(src, dst):
        if dst == build.MARSHAL:
            raise KeyboardInterrupt
        real(src, dst)

    monkeypatch.setattr(build.os, "replace", cut)
    with pytest.raises(KeyboardInterrupt):
        build.build_library(force=True)
    assert not build.marshal_fits_torch()


def test_rope_rows_kept_by_a_program_follow_the_batch(paged_batch, P, monkeypatch):
    """A tensor taken from rope_row_dev once moves with reset_decode and
    advance; lengths that the program moves, or puts in place of the batch's,
    show when the rows are next asked for."""
    rb, _, _ = paged_batch

    class Here:   # the host has no streams
        def __init__(self, *a): pass
        def __enter__(self): pass
        def __exit__(self, *a): pass

    monkeypatch.setattr(torch.cuda, "current_stream", lambda: None)
    monkeypatch.setattr(torch.cuda, "stream", Here)
    monkeypatch.setattr(P.pipeline.B, "c2kv_seq_advance", lambda t, d, s: t.add_(d))
    row = rb.rope_row_dev
    assert row.tolist() == [0, rb.cap]
    rb.reset_decode()
    assert rb.n_cached_dev.tolist() == [13, 13] and row.tolist() == [13, rb.cap + 13]
    rb.advance()
    assert rb.n_cached_dev.tolist() == [14, 14] and row.tolist() == [14, rb.cap + 14]
    rb.n_cached_dev.sub_(1)
    assert rb.rope_row_dev.tolist() == [13, rb.cap + 13]
    rb.n_cached_dev = torch.tensor([3, 5], dtype=torch.int32)
    rb.advance()
    assert rb.n_cached_dev.tolist() == [4, 6] and rb.rope_row_dev.tolist() == [4, rb.cap + 6]
    rb.reset_decode()
    assert rb.n_cached_dev.tolist() == [13, 13]
