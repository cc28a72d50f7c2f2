"""The 8-bit paged cache (filling, appending, attending) and the token log
probabilities against the fp64 oracle (oracle/pages8_oracle.py).

Bars.  Codes and scales: equal.  The rotated key is the exact rotation rounded
to fp32 and then to bf16 (the RoPE table holds cos and sin to 2^-48, so the
kernel's value before the first rounding is exact to 2^-44), the scaling is by a
power of two and the code is one rounding, so there is nothing to be off by.
Attention: the output's own bf16 rounding, 2^-8 |ref|, and the kernel's error:
its logits are off by at most ds = 2^-14 max|q| sum_i|K_ji| / sqrt(d) (the
query is held to 2^-15 of its largest element, fp32 sums on top), which moves
a convex mean of V by at most 2 ds max|V|, and its weights are off by at most
2^-11 relative: (2 ds + 2^-11) max|V|.
Log probabilities: fp32 sums of up to 2^18 terms over threads (a tree: error
below 2^-18 relative) and a difference of two numbers of at most |x|max: 2^-17
+ 2^-22 max|x|.
"""
import numpy as np
import pytest
import torch

import oracle.c2kv_oracle as O
import oracle.pages8_oracle as Q
import compressed_composable_kv_gb300 as P
from compressed_composable_kv_gb300 import synth as S
from gpu_util import to_bits, to_dev

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


class Pool:
    """A page pool on the device and its oracle copy; pages in shuffled order,
    with some that no sequence uses, codes of all kinds in every place that
    holds no row (they must neither be read nor written)."""

    def __init__(self, g, page, rows, seed=0, spare=3, extra_pages=1):
        rng = np.random.default_rng(seed)
        self.g, self.page, self.rng = g, page, rng
        counts = [max(0, -(-n // page)) for n in rows]
        self.n_pages = sum(counts) + spare
        ids = rng.permutation(self.n_pages)
        self.max_pages = max(1, max(counts) + extra_pages)
        self.table = np.full((len(rows), self.max_pages), -7, np.int32)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = ids[at:at + c]
            at += c
        shape = (g.n_layers, self.n_pages, g.n_kv_heads, page, g.head_dim)
        self.codes = [rng.integers(0, 256, shape, dtype=np.uint8) for _ in range(2)]
        self.scales = [np.exp2(rng.integers(-12, 3, shape[:3])).astype(np.float32) for _ in range(2)]
        self.upload()

    def upload(self):
        self.k8, self.v8 = (torch.from_numpy(c.copy()).cuda().view(E4) for c in self.codes)
        self.ks, self.vs = (torch.from_numpy(s.copy()).cuda() for s in self.scales)
        self.page_table = torch.from_numpy(self.table).cuda()

    def put(self, layer, b, first, kv, x):
        Q.put(self.codes[kv][layer], self.scales[kv][layer], self.page, self.table[b], first, x)

    def check(self, what):
        for name, dev, ref in (("K", self.k8, self.codes[0]), ("V", self.v8, self.codes[1])):
            got = dev.view(torch.uint8).cpu().numpy()
            a, b = Q.e4m3_values(got), Q.e4m3_values(ref)   # by value: a zero's sign is nobody's
            off = int((~((a == b) | (np.isnan(a) & np.isnan(b)))).sum())
            assert off == 0, f"{what}: {name} codes differ in {off} places"
        for name, dev, ref in (("K", self.ks, self.scales[0]), ("V", self.vs, self.scales[1])):
            off = int((dev.cpu().numpy() != ref).sum())
            assert off == 0, f"{what}: {off} {name} scales differ"

    def args(self):
        return self.k8, self.v8, self.ks, self.vs, self.page_table


def _values(rng, shape, kind="normal"):
    x = S.normal_bf16(rng, shape)
    f = O.bf16_to_f64(x)
    if kind == "wild":   # channels and rows far apart in size, zeros, subnormals, the largest numbers
        f = f * np.exp2(rng.integers(-30, 30, shape[-1]))
        f[..., 0] = 0.0
        f.reshape(-1)[:: 97] = 3.0e38
        f.reshape(-1)[5:: 211] = 1e-40
    if kind == "nan":
        f.reshape(-1)[:: 131] = np.nan
        f.reshape(-1)[7:: 173] = np.inf
        f.reshape(-1)[11:: 179] = -np.inf
    if kind == "zero":
        f = f * 0.0
    return O.f64_to_bf16(f) if kind in ("normal", "zero", "wild") else \
        torch.from_numpy(f).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def _dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def _f64(bits):
    return (np.ascontiguousarray(bits).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def _geom(d=128, group=4, n_kv=2, layers=1):
    return S.Geometry(layers, group * n_kv, n_kv, d, 5.0e5)


def _rope(g, positions):
    """Table rows of these positions, in this order, on the device."""
    pos = torch.tensor(np.asarray(positions, np.int32).reshape(-1)).cuda()
    tab = torch.empty(pos.numel() * (g.head_dim // 2) * 4, device="cuda")
    P.c2kv_rope_table(g, pos, tab)
    return tab


def _rotate(g, x, pos):
    """fp64 rotation of x [rows][heads][d] at pos[rows]."""
    h = g.head_dim // 2
    ang = np.asarray(pos, np.float64)[:, None] * g.rope_theta ** (-2.0 * np.arange(h) / g.head_dim)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = x[..., :h], x[..., h:]
    with np.errstate(invalid="ignore"):
        return np.concatenate([a * c - b * s, b * c + a * s], -1)


def _round_key(x):
    """To fp32, then to bf16; a pair with a member that is not finite is not finite."""
    h = x.shape[-1] // 2
    bad = ~np.isfinite(x[..., :h]) | ~np.isfinite(x[..., h:])
    bad = np.concatenate([bad, bad], -1)
    y = O.bf16_to_f64(O.f64_to_bf16(np.where(bad, 0.0, x).astype(np.float32).astype(np.float64)))
    return np.where(bad, np.nan, y)


def _ok():
    torch.cuda.synchronize()
    assert P.c2kv_device_error() == P.C2KV_OK


# ------------------------------------------------------------------ fill

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("kind", ["normal", "wild", "nan", "zero"])
def test_fill(d, page, kind):
    rows = [1, page - 1, 0, page, page + 1, 300, 127, 129][: 4 if kind != "normal" else 8] + [257]
    g = _geom(d, 1, 3, layers=3)
    pool = Pool(g, page, rows, seed=d + page)
    cap = 320
    k, v = ([_values(pool.rng, (3, 3, cap, d), kind) for _ in rows] for _ in range(2))
    P.c2kv_pages8_fill(g, 1, 3, [_dev(x) for x in k], [_dev(x) for x in v], cap, rows, *pool.args())
    _ok()
    for b, n in enumerate(rows):
        for l in (1, 2):
            for kv, x in ((0, k[b]), (1, v[b])):
                f = _f64(x[l][:, :n])
                pool.put(l, b, 0, kv, f)
    pool.check(f"fill d{d} page {page} {kind}")


def test_fill_twice_and_into_a_longer_sequence():
    """Filling the same rows again changes nothing; filling more rows rewrites
    the last page by its new rows' scale."""
    g = _geom(128, 4, 2)
    pool = Pool(g, 64, [200])
    k, v = (_values(pool.rng, (1, 2, 256, 128)) for _ in range(2))
    for n in (100, 100, 170):
        P.c2kv_pages8_fill(g, 0, 1, [_dev(k)], [_dev(v)], 256, [n], *pool.args())
        for kv, x in ((0, k), (1, v)):
            pool.put(0, 0, 0, kv, _f64(x[0][:, :n]))
        _ok()
        pool.check(f"fill to {n}")


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("t_len,ragged", [(1, False), (1, True), (7, True), (130, True), (300, False)])
def test_append(d, page, t_len, ragged):
    g = _geom(d, 2, 3)
    held = [0, 1, page - 1, page, 15, 127, 128, 200, -1]
    rng = np.random.default_rng(t_len + page)
    new = [int(x) for x in rng.integers(0, t_len + 1, len(held))] if ragged else [t_len] * len(held)
    new[0] = t_len
    pool = Pool(g, page, [max(0, h) + n for h, n in zip(held, new)], seed=page + t_len)
    for kv in (0, 1):   # rows held so far, of very different sizes from page to page and small ones among them
        for b, h in enumerate(held):
            if h > 0:
                pool.put(0, b, 0, kv, _f64(_values(pool.rng, (3, h, d))) * np.exp2(pool.rng.integers(-20, 3, (1, h, 1))))
    pool.upload()
    k, v = (_values(pool.rng, (len(held), t_len, 3, d)) for _ in range(2))
    start = pool.rng.integers(0, 131072 - t_len, len(held))
    pos = start[:, None] + np.arange(t_len)
    tab = _rope(g, pos)
    row = torch.arange(len(held), dtype=torch.int32, device="cuda") * t_len
    n_new = torch.tensor(new, dtype=torch.int32, device="cuda") if ragged else None
    P.c2kv_pages8_append(g, 0, *pool.args(), torch.tensor(held, dtype=torch.int32, device="cuda"), _dev(k), _dev(v), tab,
                         row, n_new)
    _ok()
    for b, (h, n) in enumerate(zip(held, new)):
        if h < 0:
            continue
        kr = _round_key(_rotate(g, _f64(k[b, :n]), pos[b, :n]))
        pool.put(0, b, h, 0, kr.transpose(1, 0, 2))
        pool.put(0, b, h, 1, _f64(v[b, :n]).transpose(1, 0, 2))
    pool.check(f"append d{d} page {page} t{t_len}")


@pytest.mark.parametrize("kind", ["wild", "nan", "zero"])
def test_append_token_by_token(kind):
    """100 single tokens onto two sequences: the scale of a page grows with
    them, and its earlier codes follow."""
    g = _geom(128, 4, 2)
    pool = Pool(g, 32, [100, 133])
    held = [0, 33]
    for kv in (0, 1):
        pool.put(0, 1, 0, kv, _f64(_values(pool.rng, (2, 33, 128))) * 2.0 ** -9)
    pool.upload()
    n_dev = torch.tensor(held, dtype=torch.int32, device="cuda")
    row = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    pos = np.concatenate([np.arange(100), 70000 + np.arange(100)])
    tab = _rope(g, pos)
    size = np.exp2(np.linspace(-12, 6, 100)) if kind != "wild" else np.ones(100)
    for t in range(100):
        k, v = (_values(pool.rng, (2, 1, 2, 128), kind) for _ in range(2))
        if kind == "nan":
            k, v = (torch.from_numpy(_f64(x) * size[t]).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
                    for x in (k, v))
        if kind == "wild":   # a rotated pair of the largest numbers may leave bf16's range on either side of it
            k, v = (O.f64_to_bf16(np.clip(_f64(x), -1e37, 1e37)) for x in (k, v))
        P.c2kv_pages8_append(g, 0, *pool.args(), n_dev, _dev(k), _dev(v), tab, row)
        P.c2kv_seq_advance(n_dev, 1)
        P.c2kv_seq_advance(row, 1)
        for b in range(2):
            kr = _round_key(_rotate(g, _f64(k[b]), [pos[100 * b + t]]))
            pool.put(0, b, held[b] + t, 0, kr.transpose(1, 0, 2))
            pool.put(0, b, held[b] + t, 1, _f64(v[b]).transpose(1, 0, 2))
    _ok()
    pool.check(f"token by token, {kind}")


@pytest.mark.parametrize("fused", [False, True])
def test_rotation_beyond_the_range_is_nan(fused):
    """Keys of the largest numbers: what the rotation takes beyond the range of
    bf16 is held as NaN, its partner and the rest as what they are."""
    g = _geom(128, 1, 2)
    pool = Pool(g, 16, [40])
    for kv in (0, 1):
        pool.put(0, 0, 0, kv, _f64(_values(pool.rng, (2, 20, 128))))
    pool.upload()
    k = _values(pool.rng, (1, 1, 2, 128))
    k[0, 0, 0, :], k[0, 0, 1, ::5] = 0x7F7F, 0xFF7F   # +- 3.39e38
    v = _values(pool.rng, (1, 1, 2, 128))
    pos = 12345
    n, row = (torch.tensor([x], dtype=torch.int32, device="cuda") for x in (20, 0))
    if fused:
        ws = torch.zeros(P.c2kv_attend_pages8_workspace_size(g, 1, 21), dtype=torch.uint8, device="cuda")
        q = torch.zeros((1, 2, 128), dtype=torch.bfloat16, device="cuda")
        P.c2kv_attend_pages8(g, 0, *pool.args(), n, 21, q, _dev(k)[:, 0], _dev(v)[:, 0], _rope(g, [pos]), row,
                             torch.empty_like(q), ws)
    else:
        P.c2kv_pages8_append(g, 0, *pool.args(), n, _dev(k), _dev(v), _rope(g, [pos]), row)
    _ok()
    with np.errstate(over="ignore"):
        kr = _round_key(_rotate(g, _f64(k[0]), [pos]))
    kr[~np.isfinite(kr)] = np.nan
    assert np.isnan(kr).any() and np.isfinite(kr).any()
    pool.put(0, 0, 20, 0, kr.transpose(1, 0, 2))
    pool.put(0, 0, 20, 1, _f64(v[0]).transpose(1, 0, 2))
    pool.check("overflowing rotation")


# ------------------------------------------------------------------ attention

def _attend_case(g, page, held, has_new=True, sharp=1.0, seed=0, kind="normal", slack=0, layer=0, bad_tail=True):
    """Runs one step and checks the output and the pool against the oracle."""
    B, d, hkv = len(held), g.head_dim, g.n_kv_heads
    add = 1 if has_new else 0
    pool = Pool(g, page, [max(0, n) + add if n >= 0 else 0 for n in held], seed=seed)
    rng = pool.rng
    for kv in (0, 1):
        for b, n in enumerate(held):
            if n > 0:
                grow = np.exp2(rng.integers(-6, 7, (1, n, 1))) if kind == "uneven" else 1.0
                pool.put(layer, b, 0, kv, _f64(_values(rng, (hkv, n, d))) * grow)
    pool.upload()
    q = S.normal_bf16(rng, (B, g.n_q_heads, d), sharp)
    k, v = (S.normal_bf16(rng, (B, hkv, d)) for _ in range(2))
    pos = rng.integers(0, 131072, B)
    tab = _rope(g, pos)
    row = torch.arange(B, dtype=torch.int32, device="cuda")
    n_dev = torch.tensor(held, dtype=torch.int32, device="cuda")
    most = max(1, max(held) + add) + slack
    ws = torch.zeros(P.c2kv_attend_pages8_workspace_size(g, B, most), dtype=torch.uint8, device="cuda")
    out = torch.full((B, g.n_q_heads, d), 7.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):   # the second call finds the token in place and the workspace used
        P.c2kv_attend_pages8(g, layer, *pool.args(), n_dev, most, _dev(q), _dev(k) if has_new else None,
                             _dev(v) if has_new else None, tab, row, out, ws)
    _ok()
    if has_new:
        for b, n in enumerate(held):
            if n >= 0:
                kr = _round_key(_rotate(g, _f64(k[b])[None], [pos[b]]))[0]
                pool.put(layer, b, n, 0, kr[:, None])
                pool.put(layer, b, n, 1, _f64(v[b])[:, None])
    pool.check("attend: pool")
    got = out.float().cpu().numpy().astype(np.float64)
    for b, n in enumerate(held):
        if n < 0:
            assert (got[b] == 7.0).all(), "an empty place of the batch was written"
            continue
        K, V = (Q.held(pool.codes[i][layer], pool.scales[i][layer], page, pool.table[b], n + add) for i in (0, 1))
        qr = _rotate(g, _f64(q[b])[None], [pos[b]])[0]
        ref = Q.attend(qr, K, V)
        if n + add == 0:
            assert (got[b] == 0).all()
            continue
        ds = 2.0 ** -14 * np.abs(qr).max() * np.abs(K).sum(-1).max() / np.sqrt(d)
        tol = 2.0 ** -8 * np.abs(ref) + (2 * ds + 2.0 ** -11) * np.abs(V).max()
        err = np.abs(got[b] - ref)
        assert np.isfinite(got[b]).all()
        assert (err <= tol).all(), f"sequence {b} of {n} rows: off by {(err - tol).max():.3e} over its bar of {tol.max():.3e}"
        # errors of either sign: their mean stays well under the worst case
        assert err.mean() <= 2.0 ** -8 * np.abs(ref).mean() + (2 * ds + 2.0 ** -11) * np.abs(V).max() / 8
    assert (ws[: 256 * hkv * 4].view(torch.int32) == 0).all(), "counters are not back at zero"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 4, 5, 8])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_attend_shapes(d, group, page):
    _attend_case(_geom(d, group, 2), page, [0, 1, 15, 16, page - 1, page, 127, 128, 129, 255, 256, 257, 700, -1],
                 seed=d + group + page)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("has_new", [True, False])
@pytest.mark.parametrize("held", [[0], [1], [3000], [5000, 0, 64], [-1, -1, 40], [-1], [1] * 64,
                                  list(range(0, 256)), [2500] + [3] * 30])
def test_attend_batches(d, has_new, held):
    _attend_case(_geom(d, 4, 2), 32, held, has_new, seed=len(held))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind,sharp", [("normal", 4.0), ("uneven", 1.0), ("uneven", 0.1)])
def test_attend_sharp_and_uneven_pages(d, kind, sharp):
    _attend_case(_geom(d, 4, 2), 16, [900, 90, 33], sharp=sharp, kind=kind)
    _attend_case(_geom(d, 8, 1), 128, [900, 90, 33], sharp=sharp, kind=kind)


def test_advance_of_a_large_batch():
    n = torch.arange(-3, 297, dtype=torch.int32, device="cuda")
    P.c2kv_seq_advance(n, 2)
    assert torch.equal(n.cpu(), torch.arange(-1, 299, dtype=torch.int32))


def test_attend_second_layer_and_generous_bound():
    _attend_case(_geom(128, 4, 8, layers=2), 64, [640, 100], layer=1, slack=50)
    _attend_case(_geom(64, 5, 1, layers=2), 64, [640, 100], layer=1, slack=50)


@pytest.mark.parametrize("n_kv,batch", [(8, 1), (8, 4), (1, 1), (40, 2)])
def test_attend_long(n_kv, batch):
    _attend_case(_geom(128, 2, n_kv), 64, [9000 - 1000 * b for b in range(batch)])
    _attend_case(_geom(64, 1, n_kv), 16, [4000 - 1000 * b for b in range(batch)])


@pytest.mark.parametrize("d,group", [(64, 1), (64, 8), (128, 4), (128, 5), (128, 8)])
@pytest.mark.parametrize("page", [16, 128])
def test_attend_more_units_than_ctas(d, group, page):
    """Every CTA's range of tiles spans several units and ends inside others."""
    rng = np.random.default_rng(d + group + page)
    lens = [int(x) for x in np.exp(rng.uniform(0.0, np.log(1800.0), 47))] + [0, -1, 1500, 256, 255]
    _attend_case(_geom(d, group, 8), page, lens, seed=group)


def test_attend_output_at_any_element():
    """out starts at an odd element; one sequence has rows, one has none."""
    g = S.Geometry(1, 4, 2, 128, 1e4)
    k8 = torch.zeros((1, 2, 2, 16, 128), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    sc = torch.ones((1, 2, 2), device="cuda")
    v8 = torch.full((1, 2, 2, 16, 128), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)   # 1.0
    table = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    n = torch.tensor([5, 0], dtype=torch.int32, device="cuda")
    q = torch.randn(2, 4, 128, device="cuda").to(torch.bfloat16)
    buf = torch.full((2 * 4 * 128 + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[1:1 + 2 * 4 * 128].view(2, 4, 128)
    rope = torch.zeros((16, 64, 4), device="cuda")
    ws = torch.zeros(P.c2kv_attend_pages8_workspace_size(g, 2, 16), dtype=torch.uint8, device="cuda")
    P.c2kv_attend_pages8(g, 0, k8, v8, sc, sc, table, n, 16, q, None, None, rope, torch.zeros_like(n), out, ws)
    assert P.c2kv_device_error() == P.C2KV_OK
    assert (out[0] == 1.0).all() and (out[1] == 0.0).all()
    assert buf[0] == 7.0 and (buf[-8:] == 7.0).all()


def test_many_faint_rows_keep_their_weight():
    """One row with weight 1 and 20000 rows of 2^-14 each, their V all ones:
    the faint rows make up over half of the answer."""
    g = _geom(128, 1, 1)
    n = 20001
    pool = Pool(g, 128, [n])
    q = np.zeros((1, 1, 128))
    q[0, 0, 0] = np.sqrt(128.0)
    x = np.zeros((1, n, 128))
    x[0, 0, 0] = 14 * np.log(2.0)          # about: the held code decides
    v = np.ones((1, n, 128))
    v[0, 0] = -1.0
    pool.put(0, 0, 0, 0, x)
    pool.put(0, 0, 0, 1, v)
    pool.upload()
    out = torch.zeros((1, 1, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(P.c2kv_attend_pages8_workspace_size(g, 1, n), dtype=torch.uint8, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    qb = O.f64_to_bf16(q)
    P.c2kv_attend_pages8(g, 0, *pool.args(), torch.tensor([n], dtype=torch.int32, device="cuda"), n, _dev(qb), None, None,
                         _rope(g, [0]), zero, out, ws)
    _ok()
    K, V = (Q.held(pool.codes[i][0], pool.scales[i][0], 128, pool.table[0], n) for i in (0, 1))
    ref = Q.attend(_f64(qb)[0], K, V)
    assert abs(ref[0, 0]) < 0.3   # neither side alone
    ds = 2.0 ** -14 * np.abs(q).max() * np.abs(K).sum(-1).max() / np.sqrt(128)
    assert np.abs(out.float().cpu().numpy()[0] - ref).max() <= 2.0 ** -8 * abs(ref).max() + (2 * ds + 2.0 ** -11)


def test_nan_rows_show_and_stay_with_their_head():
    """A NaN in one kv head's K or V: that head's queries answer NaN (V: in its
    own column), every other head as without it."""
    g = _geom(128, 4, 2)
    for kv in (0, 1):
        pool = Pool(g, 32, [70])
        for i in (0, 1):
            x = _f64(_values(pool.rng, (2, 70, 128)))
            if i == kv:
                x[1, 50, 3] = np.nan
            pool.put(0, 0, 0, i, x)
        pool.upload()
        out = torch.zeros((1, 8, 128), dtype=torch.bfloat16, device="cuda")
        ws = torch.zeros(P.c2kv_attend_pages8_workspace_size(g, 1, 70), dtype=torch.uint8, device="cuda")
        zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        P.c2kv_attend_pages8(g, 0, *pool.args(), torch.tensor([70], dtype=torch.int32, device="cuda"), 70,
                             _dev(S.normal_bf16(pool.rng, (1, 8, 128))), None, None, _rope(g, [5]), zero, out, ws)
        _ok()
        nan = out.isnan()[0].cpu()
        assert not nan[:4].any()
        assert nan[4:].all() if kv == 0 else (nan[4:, 3].all() and nan[4:].sum() == 4)


# ------------------------------------------------------------------ device-side checks

def test_bad_device_values_are_reported_and_left_out():
    """A length above max_keys, a page id outside the pool, a table row outside
    the table: the error word says so, the sequence (or the page) is left out,
    its neighbours are served and the workspace is usable again."""
    g = _geom(128, 4, 2)
    pool = Pool(g, 32, [101, 101, 101])
    for kv in (0, 1):
        for b in range(3):
            pool.put(0, b, 0, kv, _f64(_values(pool.rng, (2, 100, 128))))
    pool.upload()
    ws = torch.zeros(P.c2kv_attend_pages8_workspace_size(g, 3, 101), dtype=torch.uint8, device="cuda")
    q = _dev(S.normal_bf16(pool.rng, (3, 8, 128)))
    kn, vn = (_dev(S.normal_bf16(pool.rng, (3, 2, 128))) for _ in range(2))
    tab = _rope(g, [9, 10, 11])
    rows = torch.arange(3, dtype=torch.int32, device="cuda")

    def step(held=(100, 100, 100), row=rows, table=pool.page_table):
        out = torch.full((3, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        P.c2kv_attend_pages8(g, 0, pool.k8, pool.v8, pool.ks, pool.vs, table,
                             torch.tensor(held, dtype=torch.int32, device="cuda"), 101, q, kn, vn, tab, row, out, ws)
        torch.cuda.synchronize()
        return out, P.c2kv_device_error()

    good, code = step()
    assert code == P.C2KV_OK
    for held, row in (((100, 101, 100), rows), ((100, 100, 100), torch.tensor([0, 3, 2], dtype=torch.int32, device="cuda")),
                      ((100, 100, 100), torch.tensor([0, -1, 2], dtype=torch.int32, device="cuda"))):
        out, code = step(held, row)
        assert code == P.C2KV_EDEVICE
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
        assert (out[1] == 7.0).all()
    for bad in (-1, pool.n_pages, 2 ** 31 - 1):
        table = pool.page_table.clone()
        table[1, 1] = bad
        out, code = step(table=table)
        assert code == P.C2KV_EDEVICE
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    out, code = step()
    assert code == P.C2KV_OK and torch.equal(out, good)


def test_append_leaves_out_what_does_not_fit():
    g = _geom(64, 1, 2)
    pool = Pool(g, 16, [40, 40, 40], extra_pages=0)
    tab = _rope(g, np.arange(12))
    kn, vn = (_dev(S.normal_bf16(pool.rng, (3, 4, 2, 64))) for _ in range(2))
    pool_rows = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    for held, new, row in (([46, 46, 46], None, pool_rows),                       # past max_pages
                           ([0, 0, 0], [5, -1, 5], pool_rows),                    # not in [0, t_len]
                           ([0, 0, 0], None, pool_rows + 12)):                    # past the table
        P.c2kv_pages8_append(g, 0, *pool.args(), torch.tensor(held, dtype=torch.int32, device="cuda"), kn, vn, tab, row,
                             None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert P.c2kv_device_error() == P.C2KV_EDEVICE
        pool.check("nothing written")


# ------------------------------------------------------------------ log probabilities

def _logprobs(x, tokens, k, stream=None):
    rows = x.shape[0]
    lp, ent = torch.full((rows,), 5.0, device="cuda"), torch.full((rows,), 5.0, device="cuda")
    ids = torch.full((rows, k), -5, dtype=torch.int32, device="cuda")
    tops = torch.full((rows, k), 5.0, device="cuda")
    P.c2kv_token_logprobs(x, tokens, k, lp if tokens is not None else None, ent, ids, tops, stream)
    torch.cuda.synchronize()
    return lp, ent, ids, tops


def _check_logprobs(x, k, seed=0, tokens=None):
    rng = np.random.default_rng(seed)
    rows, vocab = x.shape
    if tokens is None:
        tokens = rng.integers(-1, vocab, rows).astype(np.int32)
    lp, ent, ids, tops = _logprobs(x, torch.from_numpy(tokens).cuda(), k)
    assert P.c2kv_device_error() == P.C2KV_OK
    xf = x.double().cpu().numpy()
    r_lp, r_ent, r_ids, r_tops = Q.token_logprobs(xf, tokens, k)
    assert np.array_equal(ids.cpu().numpy(), r_ids)
    size = np.abs(xf)
    size[~(size < 1e30)] = 0.0   # masks
    tol = 2.0 ** -17 + 2.0 ** -22 * size.max(-1)
    for got, ref in ((lp, r_lp), (ent, r_ent), (tops, r_tops)):
        got = got.double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(np.isneginf(got), np.isneginf(ref))
        fine = np.isfinite(ref)
        bar = (tol if ref.ndim == 1 else tol[:, None]) + 2.0 ** -22 * np.where(fine, np.abs(ref), 0.0)
        assert np.all(np.abs(np.where(fine, got, 0.0) - np.where(fine, ref, 0.0)) <= bar)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (2, 7), (5, 1000), (4, 128256), (1, 151936), (2, 50257),
                                        (300, 8191), (33, 32769), (1, 600001)])
@pytest.mark.parametrize("k", [0, 1, 20])
def test_logprobs(dtype, rows, vocab, k):
    gen = torch.Generator(device="cuda").manual_seed(rows + vocab)
    x = (torch.randn(rows, vocab, generator=gen, device="cuda") * 3).to(dtype)
    _check_logprobs(x, min(k, vocab))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [64, 5001, 128256])
def test_logprobs_ties_masks_and_strange_rows(dtype, vocab):
    """All equal; few different values; nearly all ruled out; all ruled out; the
    type's lowest value as a mask; very large logits; NaN and +inf; -0 and +0."""
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    x = torch.randn(12, vocab, generator=gen, device="cuda")
    x[0] = 0.25
    x[1] = (x[1] > 0).float()
    x[2, :] = -torch.inf
    x[2, vocab // 2] = 3.0
    x[2, vocab - 1] = 1.0
    x[3] = -torch.inf
    x[4, : vocab - 3] = torch.finfo(dtype).min
    x[5] = x[5] * 1e4
    x[6, vocab // 3] = torch.nan
    x[7, vocab // 5] = torch.inf
    x[8] = torch.where(x[8] > 0, 0.0, -0.0)
    x[9] = torch.arange(vocab, device="cuda") / 8.0
    x[10] = -torch.arange(vocab, device="cuda") / 8.0
    x[11] = torch.finfo(dtype).min
    _check_logprobs(x.to(dtype), 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [200, 40000, 300007])
@pytest.mark.parametrize("k", [1, 20, 64])
def test_logprobs_of_many_equal_and_unordered_logits(dtype, vocab, k):
    """NaN everywhere, in most places, from the second logit on; +inf in most
    places; masks that leave a range at the end, every 50th token, a random
    tenth; equal logits but for a few larger ones late in the row; logits that
    rise along the row, smoothly and by steps; parts of every 2048 ruled out."""
    gen = torch.Generator(device="cuda").manual_seed(vocab + k)
    x = torch.randn(13, vocab, generator=gen, device="cuda")
    few = torch.rand(vocab, generator=gen, device="cuda") < 0.1
    x[0] = torch.nan
    x[1, ~few] = torch.nan
    x[2, 1:] = torch.nan
    x[3, ~few] = torch.inf
    x[4, : vocab - vocab // 3] = -torch.inf
    x[5, : vocab - vocab // 3] = torch.finfo(dtype).min
    x[6, torch.arange(vocab, device="cuda") % 50 != 7] = torch.finfo(dtype).min
    x[7, ~few] = -torch.inf
    x[8] = 1.0
    x[8, vocab - 30 :: 7] = 2.0
    x[9] = torch.arange(vocab, device="cuda") / 1000.0
    x[10] = torch.arange(vocab, device="cuda") // 5000 + x[10].clamp(-0.4, 0.4)
    x[11, torch.arange(vocab, device="cuda") % 2048 < 64] = -100.0   # some of a step's groups far below the others
    x[12, (torch.arange(vocab, device="cuda") % 1024 < 32) | ~few] = -torch.inf
    _check_logprobs(x.to(dtype), k)


def test_logprobs_strides_offsets_and_options():
    """Rows an odd stride apart, starting at any element; outputs that are not
    asked for; a token outside the vocabulary."""
    base = torch.randn(6 * 10007 + 9, device="cuda")
    for dtype in (torch.bfloat16, torch.float32):
        b = base.to(dtype)
        for off in range(9):
            x = b[off:off + 6 * 10007].view(6, 10007)[:, :9001]
            _check_logprobs(x, 5, seed=off)
    x = base[:20000].view(2, 10000)
    lp, ent, ids, tops = _logprobs(x, None, 3)
    assert (lp == 5.0).all() and (ent != 5.0).all()
    top = torch.full((2, 3), 5.0, device="cuda")
    P.c2kv_token_logprobs(x, None, 0, None, None)
    only = torch.zeros(2, device="cuda")
    P.c2kv_token_logprobs(x, torch.tensor([1, 2], dtype=torch.int32, device="cuda"), 0, only, None)
    assert torch.allclose(only, torch.log_softmax(x, -1)[[0, 1], [1, 2]], atol=1e-5) and (top == 5.0).all()
    lp, *_ = _logprobs(x, torch.tensor([10000, 3], dtype=torch.int32, device="cuda"), 0)
    assert lp[0].isnan() and not lp[1].isnan()
    assert P.c2kv_device_error() == P.C2KV_EDEVICE


def test_wrong_device_tensors_are_refused():
    x = torch.zeros((2, 10), device="cuda")
    with pytest.raises(ValueError, match="current CUDA device"):
        P.c2kv_token_logprobs(x, torch.zeros(2, dtype=torch.int32), 0, torch.zeros(2, device="cuda"), None)


def test_offsets_beyond_32_bits():
    """Pages 4 GB and more into their pool, in the second layer, and rows of
    logits beyond 2^31 elements: as in a small pool, as on their own."""
    g = S.Geometry(2, 16, 8, 128, 1e4)
    t_len, page, many = 300, 128, 20000      # 128 KB a page, 2.6 GB a layer
    ids = torch.tensor([many - 1, many - 3, many - 2], dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(5)
    kn, vn = (_dev(S.normal_bf16(rng, (1, t_len, 8, 128))) for _ in range(2))
    k1, v1 = (_dev(S.normal_bf16(rng, (1, 8, 128))) for _ in range(2))
    q = _dev(S.normal_bf16(rng, (1, 16, 128)))
    tab = _rope(g, np.arange(t_len + 1))
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    caches = [torch.randn(2, 8, 320, 128, device="cuda").to(torch.bfloat16) for _ in range(2)]
    got = []
    for n, table in ((many, ids[None]), (3, torch.arange(3, dtype=torch.int32, device="cuda")[None])):
        k8, v8 = (torch.empty((2, n, 8, page, 128), dtype=E4, device="cuda") for _ in range(2))
        ks, vs = (torch.empty((2, n, 8), device="cuda") for _ in range(2))
        table = table.contiguous()
        at = table[0].long()
        for t in (k8, v8):
            t[1].view(torch.uint8)[at] = 0
        pool = (k8, v8, ks, vs, table)
        P.c2kv_pages8_append(g, 1, *pool, zero, kn, vn, tab, zero)
        ws = torch.zeros(P.c2kv_attend_pages8_workspace_size(g, 1, t_len + 1), dtype=torch.uint8, device="cuda")
        out = torch.empty((1, 16, 128), dtype=torch.bfloat16, device="cuda")
        P.c2kv_attend_pages8(g, 1, *pool, zero + t_len, t_len + 1, q, k1, v1, tab, zero + t_len, out, ws)
        res = [out.float()] + [t[1].view(torch.uint8)[at] for t in (k8, v8)] + [t[1][at] for t in (ks, vs)]
        P.c2kv_pages8_fill(g, 0, 2, caches[:1], caches[1:], 320, [257], *pool)
        got.append(res + [t[1].view(torch.uint8)[at] for t in (k8, v8)] + [t[1][at] for t in (ks, vs)])
        _ok()
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert got[0][0].isfinite().all() and got[0][0].abs().max() > 0
    del got, pool, k8, v8
    x = torch.empty((18000, 128256), dtype=torch.bfloat16, device="cuda")
    x[:] = torch.randn(128256, device="cuda").to(torch.bfloat16)
    x[-1] = x[-1].flip(0)
    tok = torch.full((18000,), 77, dtype=torch.int32, device="cuda")
    all_rows, last = _logprobs(x, tok, 4), _logprobs(x[-1:].clone(), tok[:1], 4)
    for a, b in zip(all_rows, last):
        # sums of the row in another order: a few fp32 roundings of values below 32
        assert (a[-1:].double() - b.double()).abs().max() <= 2.0 ** -17
        assert torch.equal(a[0], a[-2])


def test_table_rows_at_the_lengths():
    """C2KV_DECODE_ROW_AT_LENGTH: the table row is rope_row_dev[b] +
    n_cached_dev[b] (from a negative start too); the sum is checked."""
    g = _geom(128, 4, 2)
    held, place = [100, 7, 0, -1], [3, 300, 500, 5]
    pool = Pool(g, 32, [n + 1 for n in held])
    for kv in (0, 1):
        for b, n in enumerate(held):
            if n > 0:
                pool.put(0, b, 0, kv, _f64(_values(pool.rng, (2, n, 128))))
    q = _dev(S.normal_bf16(pool.rng, (4, 8, 128)))
    kn, vn = (_dev(S.normal_bf16(pool.rng, (4, 2, 128))) for _ in range(2))
    tab = _rope(g, np.arange(512))
    n_dev = torch.tensor(held, dtype=torch.int32, device="cuda")
    ws = torch.zeros(P.c2kv_attend_pages8_workspace_size(g, 4, 101), dtype=torch.uint8, device="cuda")

    def step(rows, flags):
        pool.upload()
        out = torch.full((4, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        P.c2kv_attend_pages8(g, 0, *pool.args(), n_dev, 101, q, kn, vn, tab,
                             torch.tensor(rows, dtype=torch.int32, device="cuda"), out, ws, flags=flags)
        torch.cuda.synchronize()
        return [out] + [t.view(torch.uint8).clone() for t in pool.args()[:4]], P.c2kv_device_error()

    want, code = step(place, 0)
    assert code == P.C2KV_OK
    got, code = step([p - n for p, n in zip(place, held)], P.C2KV_DECODE_ROW_AT_LENGTH)
    assert code == P.C2KV_OK and all(torch.equal(a, b) for a, b in zip(want, got))
    for bad in (512 - 100, -101, 2 ** 31 - 1, -2 ** 31):
        got, code = step([bad] + [p - n for p, n in zip(place[1:], held[1:])], P.C2KV_DECODE_ROW_AT_LENGTH)
        assert code == P.C2KV_EDEVICE
        assert (got[0][0] == 7.0).all() and torch.equal(got[0][1:], want[0][1:])
