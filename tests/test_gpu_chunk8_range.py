"""Chunk attention over the 8-bit pages at the ends of its range, against the fp64
oracle (oracle/pages8_oracle.py): units of one tile, many to a CTA; pages whose scales
are far apart."""
import numpy as np
import pytest
import torch

import oracle.pages8_oracle as Q
from test_gpu_chunk8 import Chunk
from test_gpu_pages8 import _f64, _geom, _ok, _rotate, _values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t_len,held", [(3, 110), (3, 330), (60, 60)])
def test_many_units_of_few_tiles(t_len, held):
    """2048 units of one to three tiles, 13 and more to a CTA: the places in shared memory
    that describe a tile serve again and again, and every other unit leaves one of the two
    MMA issuers nothing to do."""
    g = _geom(64, 2, 8)
    c = Chunk(g, 16, [(i * 37) % held for i in range(256)], [1 + i % t_len for i in range(256)], t_len=t_len, seed=t_len + held)
    want = c.call().clone()
    _ok()
    for _ in range(20):
        assert (c.call(k_new=None, v_new=None) == want).all()
    _ok()
    c.put_new()
    c.check("few tiles", rows=[0, 1, t_len - 1])


# ------------------------------------------------------------------ scales far apart

FIRST = 8.0   # element 0 of every rotated query


def _aimed(g, page, held, new, seed):
    """A chunk whose queries, once rotated, have FIRST in element 0."""
    c = Chunk(g, page, held, new, seed=seed)
    for b in range(len(held)):
        turned = c.pool.rng.standard_normal((c.t_len, g.n_q_heads, g.head_dim))
        turned[..., 0] = FIRST
        c.q[b] = _bits(_rotate(g, turned, -c.pos[b]))
    return c


def _bits(x):
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def _hold(c, b, keys, values):
    """The held rows of sequence b: [kv head][row][d]."""
    for kv, x in ((0, keys), (1, values)):
        c.pool.put(0, b, 0, kv, x)
    c.pool.upload()


def _normal_rows(c, n, size=1.0):
    shape = (c.g.n_kv_heads, n, c.g.head_dim)
    return _f64(_values(c.pool.rng, shape)), _f64(_values(c.pool.rng, shape)) * size


def _size(c, far):
    """What all values are multiplied by, so that those 2^far above are numbers, too."""
    size = 1.0 if far < 120 else 2.0 ** -60
    c.v = _bits(_f64(c.v) * size)
    return size


def _check_by_column(c, what, skip=None, rows=None):
    """Each element of the answer against what the keys' own weights and that column's own
    values may move it by: a logit is off by ds_j = (2^-11 + 2^-18) sum_i |q_i K_ji| / sqrt(d)
    (queries in fp16, sums in fp32), so numerator and denominator by ds_j p_j; a weight is
    rounded to fp16, 2^-11 of itself or, below fp16's normal range, 2^-25 of the largest
    but no more than itself; sums in fp32 add 2^-15; then the rounding to bf16, 2^-8 or
    2^-134.  1.1: products of these."""
    c.pool.check(what)
    g, pl = c.g, c.pool
    out = c.out.float().cpu().numpy().astype(np.float64)
    worst = 0.0
    for b, (h, n) in enumerate(zip(c.held, c.new)):
        k, v = (Q.held(pl.codes[x][0], pl.scales[x][0], c.page, pl.table[b], h + n) for x in (0, 1))
        q = _rotate(g, _f64(c.q[b, :n]), c.pos[b, :n])
        for i in range(n) if rows is None else sorted({r % n for r in rows}):
            for head in range(g.n_q_heads):
                kv = head // (g.n_q_heads // g.n_kv_heads)
                K, V = k[kv, :h + i + 1], v[kv, :h + i + 1]
                s = K @ q[i, head] / np.sqrt(g.head_dim)
                p = np.exp(s - s.max())
                top = 1.0 / p.sum()
                p = p * top
                ds = (2.0 ** -11 + 2.0 ** -18) * (np.abs(K) @ np.abs(q[i, head])) / np.sqrt(g.head_dim)
                ds = np.where(p > 0, ds, 0.0)
                ref = p @ V
                moved = p * (ds + p @ ds + 2.0 ** -11 + 2.0 ** -15) + np.minimum(2.0 ** -25 * top, p)
                tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -134 + 1.1 * moved @ np.abs(V)
                err = np.abs(out[b, i, head] - ref)
                if skip is not None:
                    err = np.where(skip[b, i, head], 0.0, err)
                at = int(np.argmax(np.where(err <= tol, 0.0, err)))
                assert (err <= tol).all(), f"{what}: sequence {b} token {i} head {head} column {at}: {out[b, i, head, at]:.6e}, not {ref[at]:.6e} ({err[at] / tol[at]:.1f} of the bar)"
                worst = max(worst, (err / tol).max())
    return worst


SPREADS = [(d, group, page, t, far) for d, group, t in ((128, 4, 20), (64, 2, 70), (128, 5, 60)) for page in (16, 128) for far in (6, 14, 20, 26, 33, 60, 110, 160, 180)]


@pytest.mark.parametrize("d,group,page,t,far", SPREADS)
def test_large_values_that_no_query_looks_at(d, group, page, t, far):
    """Pages whose values are 2^far of the others', and whose keys no query looks at, cost the
    other rows' answer nothing, before them, behind them or among 128 neighbouring rows."""
    g = _geom(d, group, 2)
    held = [129, 600, 1500]
    c = _aimed(g, page, held, [t] * 3, seed=far)
    size = _size(c, far)
    for b, n in enumerate(held):
        k, v = _normal_rows(c, n, size)
        for first in (0, 256, 1152)[:1 + b]:
            far_rows = slice(first, first + page)
            k[:, far_rows] = 0.0
            k[:, far_rows, 0] = -2.0 ** 13   # -5800 and less as a logit
            v[:, far_rows] *= 2.0 ** far
        _hold(c, b, k, v)
    c.call()
    _ok()
    c.put_new()
    _check_by_column(c, f"2^{far}")


@pytest.mark.parametrize("d,group,page,t,far", SPREADS)
def test_large_values_in_one_column(d, group, page, t, far):
    """Pages with 2^far in one column, which the queries look at as at any other: the other
    columns keep what the other pages put there."""
    g = _geom(d, group, 2)
    held = [128, 600, 1500]
    c = _aimed(g, page, held, [t] * 3, seed=far + 1)
    size = _size(c, far)
    for b, n in enumerate(held):
        k, v = _normal_rows(c, n, size)
        for first in (0, 256, 1152)[:1 + b]:
            v[:, first:first + page] = 0.0
            v[:, first:first + page, 7] = 2.0 ** far * size
        _hold(c, b, k, v)
    c.call()
    _ok()
    c.put_new()
    _check_by_column(c, f"2^{far}")


@pytest.mark.parametrize("d,group,page,t,far", SPREADS)
def test_large_keys_that_no_query_looks_at(d, group, page, t, far):
    """A key of 2^far that every query turns away from: logits of rows on neighbouring pages
    are as exact as ever."""
    if far > 60:   # the logit itself stays in fp32's range
        far = 80
    g = _geom(d, group, 2)
    held = [129, 600]
    c = _aimed(g, page, held, [t] * 2, seed=far + 2)
    for b, n in enumerate(held):
        k, v = _normal_rows(c, n)
        k[:, page:, 1] *= 4.0
        for first in (0, 512)[:1 + b]:
            k[:, first] = 0.0
            k[:, first, 0] = -2.0 ** far
        _hold(c, b, k, v)
    c.call()
    _ok()
    c.put_new()
    _check_by_column(c, f"2^{far}")


@pytest.mark.parametrize("size", [2.0 ** 124, 2.0 ** -112])
@pytest.mark.parametrize("held,new", [([300, 40], [20, 20]), ([6000, 3], [3, 40]), ([3000], [300])])
def test_values_at_the_ends_of_the_range(size, held, new):
    """Values near the largest and the smallest that a page holds, units cut and whole: the
    answer is a mean of them, and so in range, at every step on the way to it."""
    g = _geom(128, 4, 2)
    c = Chunk(g, 64, held, new, t_len=max(new), seed=31)
    for b, n in enumerate(held):
        k, v = _normal_rows(c, n)
        _hold(c, b, k, np.clip(v, -2.5, 2.5) * size)
        c.v[b] = _bits(np.clip(_f64(c.v[b]), -2.5, 2.5) * size)
    c.call()
    _ok()
    c.put_new()
    _check_by_column(c, "ends")


@pytest.mark.parametrize("d,page", [(128, 16), (64, 32), (128, 64)])
@pytest.mark.parametrize("t", [1, 9, 70])
def test_pages_of_every_scale(d, page, t):
    """Neighbouring pages of all sizes, pages of zeros among them, NaN that some tokens see."""
    g = _geom(d, 4, 2)
    held = [0, 129, 700]
    c = _aimed(g, page, held, [t] * 3, seed=t + page)
    rng = c.pool.rng
    for b, n in enumerate(held):
        if n:
            k, v = _normal_rows(c, n)
            pages = -(-n // page)
            k *= np.exp2(np.repeat(rng.integers(-60, 2, (2, pages)), page, 1)[:, :n, None])
            size = np.repeat(rng.choice([-100, -40, -14, -3, 0, 0, 9, 30, 80], (2, pages)), page, 1)[:, :n, None]
            v *= np.where(np.repeat(rng.random((2, pages)) < 0.2, page, 1)[:, :n, None], 0.0, np.exp2(size))
            _hold(c, b, k, v)
    c.v[2, t // 2, 1, 3] = 0x7FC0
    c.call()
    _ok()
    c.put_new()
    out = c.out.float().cpu().numpy()
    nan = np.isnan(out)
    want = np.zeros_like(nan)
    want[2, t // 2:, 4:, 3] = True
    assert np.array_equal(nan, want)
    for x in (c.pool.codes[1], c.pool.v8.view(torch.uint8)):   # the other elements
        x[(x & 0x7F) == 0x7F] = 0
    c.out.copy_(torch.from_numpy(np.where(want, 0.0, out)))
    _check_by_column(c, "every scale", skip=want)


def test_pages_of_zeros_beside_others():
    """Pages of zeros, whose scale is the smallest there is, cost no exactness and no detour."""
    g = _geom(128, 4, 2)
    c = _aimed(g, 16, [900], [40], seed=40)
    k, v = _normal_rows(c, 900)
    v[:, 32:64], v[:, 640:656] = 0.0, 0.0
    k[:, 300:333] = 0.0
    _hold(c, 0, k, v)
    c.call()
    _ok()
    c.put_new()
    _check_by_column(c, "zeros")


@pytest.mark.parametrize("d,group,page,t,held", [
    (128, 5, 16, 70, [5000, 4990, 128, 3100]),    # units of 256 and of 94 rows, cut
    (128, 5, 128, 70, [5000, 4990, 128, 3100]),
    (64, 4, 32, 300, [2700, 129, 2700]),          # of 256 and of 176 rows
])
@pytest.mark.parametrize("kind", ["values", "column", "keys", "all"])
def test_units_of_256_rows(d, group, page, t, held, kind):
    """The same at the sizes that take 256 rows to a unit: a large value or key that no query
    looks at, one column, neighbouring pages of every scale, zeros among them."""
    g = _geom(d, group, 8)
    c = _aimed(g, page, held, [t] * len(held), seed=t + page)
    rng = c.pool.rng
    for b, n in enumerate(held):
        k, v = _normal_rows(c, n)
        pages = -(-n // page)
        if kind == "all":
            k *= np.exp2(np.repeat(rng.integers(-60, 2, (8, pages)), page, 1)[:, :n, None])
            size = np.exp2(rng.choice([-100, -40, -14, -3, 0, 0, 9, 30, 80], (8, pages))) * (rng.random((8, pages)) > 0.2)
            v *= np.repeat(size, page, 1)[:, :n, None]
        for i, first in enumerate((0, 640, 1408, 2304) if kind != "all" else ()):
            at, far = slice(first, first + page), (20, 40, 14, 100)[i]
            if kind == "values":
                k[:, at] = 0.0
                k[:, at, 0] = -2.0 ** 13
                v[:, at] *= 2.0 ** far
            elif kind == "column":
                v[:, at] = 0.0
                v[:, at, 7] = 2.0 ** far
            else:
                k[:, at] = 0.0
                k[:, at, 0] = -2.0 ** min(far, 80)
        _hold(c, b, k, v)
    c.call()
    _ok()
    c.put_new()
    _check_by_column(c, kind, rows=[0, 31, 32, 50, 51, t - 1])
