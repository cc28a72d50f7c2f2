"""Decode attention over 8-bit pages on data where every key shows.

Values: row j of head h is a power of two in one channel, the channel of its
block of keys, so an element of the output is the weight of one block of
(n + 1) / d keys, all terms positive. Weights are equal (a zero query) or
within e of each other (keys and query in channel 0, position 0, no rotation).
Keys, values and scales are exact in the pages; the query's three parts hold it
to 2^-14.8 and with it a score of at most 1, a weight's three parts hold it to
2^-12, fp32 adds less than 2^-20: below 2^-11 of an element, next to its own
rounding of 2^-8. So the bar is (2^-8 + 2^-11) |ref|, and a single key left
out or taken twice, 1/81 of its block at least with equal weights and 1/(2.8 x
47) with others, is beyond it; so are pages or scales of another place.

Random data: the query's elements are off by r, |r_i| <= 2^-14.8 max|q|, so the
scores by K r / sqrt(d) and the output, to first order, by M^T r / sqrt(d) with
M = sum_j p_j K_j (V_j - out)^T: at most 2^-14.8 max|q| |M|. What is of second
order, with e = max_j |K_j r| / sqrt(d) <= 2^-14.8 max|q| |K_j|, is at most
(exp(2 e) - 1 - 2 e + e^2) sum_j p_j |V_j - out|, and the sum of d products in
fp32 takes another (exp(2 f) - 1) of it, f = d 2^-23 sum_i |q_i K_ji| / sqrt(d).
The output's elements are held as above, a weight to 2^-12.
"""
import numpy as np
import pytest
import torch

import oracle.c2kv_oracle as O
import oracle.pages8_oracle as Q

BAR = 2.0 ** -8 + 2.0 ** -11


def keyed_rows(n, d, hkv, seq, weighted):
    """K, V [hkv][n][d] of a sequence whose every key shows."""
    j = np.arange(n)
    per = -(-n // d)
    K, V = np.zeros((hkv, n, d)), np.zeros((hkv, n, d))
    for h in range(hkv):
        block = j // per + 3 * h + 5 * seq
        V[h, j, block % d] = 2.0 ** (block % 4 - 1)
        if weighted:   # 1 .. 1.875 over a power of two that changes every 48 keys
            K[h, j, 0] = (1 + (5 * j + h) % 8 / 8) * 2.0 ** -(j // 48 % 5)
    return K, V


def keyed_query(d, hq, weighted):
    q = np.zeros((hq, d))
    if weighted:
        q[:, 0] = 0.5 * np.sqrt(d)      # scores below 1
    return O.bf16_to_f64(O.f64_to_bf16(q))


def worst(got, ref):
    """The largest error over its bar; where the reference is 0 so is the answer."""
    err = np.abs(got - ref)
    return np.where(ref > 0, err / (BAR * np.maximum(ref, 1e-30)), np.where(err > 0, np.inf, 0.0)).max()


@pytest.mark.parametrize("n,d,weighted", [(9001, 128, False), (4096, 64, False), (6001, 128, True), (2500, 64, True),
                                          (700, 128, True)])
def test_the_bar_sees_a_single_key(n, d, weighted):
    K, V = keyed_rows(n, d, 1, 0, weighted)
    q = keyed_query(d, 1, weighted)
    ref = Q.attend(q, K, V)
    assert worst(ref, ref) == 0.0
    def without(keep):
        return Q.attend(q, K[:, keep], V[:, keep])
    for at in (0, 1, n // 3, n // 2, n - 2, n - 1):
        assert worst(without(np.arange(n) != at), ref) > 1
        assert worst(without(np.sort(np.append(np.arange(n), at))), ref) > 1
    assert worst(without(np.arange(n) // 128 != n // 256), ref) > 50     # a tile
    if weighted:      # K of one 16-token page under its neighbour's power of two
        K2 = K.copy()
        K2[:, 48:64] *= 2.0
        assert worst(Q.attend(q, K2, V), ref) > 1
    V2 = V.copy()
    V2[:, 64:80] *= 2.0
    assert worst(Q.attend(q, K, V2), ref) > 10


# ------------------------------------------------------------------ on the GPU

def _run(g, pool, held, q, k, v, pos, has_new):
    import compressed_composable_kv_gb300 as P
    from test_gpu_pages8 import _dev, _ok, _rope
    batch, most = len(held), max(1, max(held) + has_new)
    ws = torch.zeros(P.c2kv_attend_pages8_workspace_size(g, batch, most), dtype=torch.uint8, device="cuda")
    out = torch.full((batch, g.n_q_heads, g.head_dim), 7.0, dtype=torch.bfloat16, device="cuda")
    n_dev = torch.tensor(held, dtype=torch.int32, device="cuda")
    row = torch.arange(batch, dtype=torch.int32, device="cuda")
    P.c2kv_attend_pages8(g, 0, *pool.args(), n_dev, most, _dev(q), _dev(k) if has_new else None,
                         _dev(v) if has_new else None, _rope(g, pos), row, out, ws)
    _ok()
    return out.double().cpu().numpy()


LENS = [[9000], [5000, 64, 0], [6000, 2999, 128, 127, 1], [15, 16, 255, 256, 257, 700], [1] * 40 + [300],
        [61 * i % 1400 for i in range(60)]]


@pytest.mark.gpu
@pytest.mark.parametrize("d,group,hkv,page", [(128, 4, 8, 64), (128, 5, 2, 16), (128, 1, 8, 128), (64, 2, 8, 32),
                                              (64, 8, 1, 16)])
@pytest.mark.parametrize("held", LENS)
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("has_new", [True, False])
def test_every_key_counts_once(d, group, hkv, page, held, weighted, has_new):
    from test_gpu_pages8 import Pool, _geom
    most = {(128, False): 10000, (128, True): 6000, (64, False): 5000, (64, True): 2900}[d, weighted]
    held = [min(n, most) for n in held]
    g = _geom(d, group, hkv)
    pool = Pool(g, page, [n + has_new for n in held], seed=page)
    rows = [keyed_rows(n + has_new, d, hkv, b, weighted) for b, n in enumerate(held)]
    for b, n in enumerate(held):
        for kv in (0, 1):
            if n > 0:
                pool.put(0, b, 0, kv, rows[b][kv][:, :n])
    pool.upload()
    q = np.stack([keyed_query(d, g.n_q_heads, weighted)] * len(held))
    new = [np.stack([O.f64_to_bf16(r[kv][:, n]) if has_new else np.zeros((hkv, d), np.uint16)
                     for r, n in zip(rows, held)]) for kv in (0, 1)]
    got = _run(g, pool, held, O.f64_to_bf16(q), *new, [0] * len(held), has_new)
    for b, n in enumerate(held):
        if n + has_new == 0:
            assert (got[b] == 0).all()
            continue
        off = worst(got[b], Q.attend(q[b], *rows[b]))
        assert off <= 1, f"sequence {b} of {n} rows: {off:.2f} of its bar"


def mean_square_bar(qr, K, V, ref):
    """Bound of |got - ref| for each query head (qr rotated, K and V as held)."""
    group, d = qr.shape[0] // K.shape[0], qr.shape[1]
    bar = np.zeros(qr.shape[0])
    for h in range(qr.shape[0]):
        k, v = K[h // group], V[h // group]
        s = k @ qr[h] / np.sqrt(d)
        p = np.exp(s - s.max())
        p /= p.sum()
        near = v - ref[h]
        r = 2.0 ** -14.8 * np.abs(qr[h]).max()
        e = r * np.linalg.norm(k, axis=-1).max()
        f = d * 2.0 ** -23 * (np.abs(k) @ np.abs(qr[h])).max() / np.sqrt(d)
        spread = (p * np.linalg.norm(near, axis=-1)).sum()
        size = (p * np.linalg.norm(v, axis=-1)).sum()
        bar[h] = (2.0 ** -8 * np.linalg.norm(ref[h]) + r * np.linalg.norm(k.T @ (p[:, None] * near)) + 2.0 ** -12 * size
                  + (np.expm1(2 * e) - 2 * e + e * e + np.expm1(2 * f)) * spread)
    return bar


@pytest.mark.gpu
@pytest.mark.parametrize("d,group", [(128, 4), (128, 5), (64, 8)])
@pytest.mark.parametrize("outlier", [1.0, 8.0, 32.0])
@pytest.mark.parametrize("held", [[8000], [900, 90, 33]])
def test_queries_with_outlying_channels(d, group, outlier, held):
    """A query with a few channels far above the others, where K's are small
    and where they are not."""
    from compressed_composable_kv_gb300 import synth as S
    from test_gpu_pages8 import Pool, _f64, _geom, _rotate, _round_key, _values
    g = _geom(d, group, 2)
    pool = Pool(g, 32, [n + 1 for n in held], seed=d + group)
    rng = pool.rng
    loud = np.ones(d)
    loud[[3, d // 2 - 1]] = outlier
    quiet = np.ones(d)
    quiet[3] = 1.0 / outlier        # one loud channel meets small keys, the other does not
    for kv in (0, 1):
        for b, n in enumerate(held):
            pool.put(0, b, 0, kv, _f64(_values(rng, (2, n, d))) * (quiet if kv == 0 else 1.0))
    pool.upload()
    B = len(held)
    q = O.f64_to_bf16(_f64(S.normal_bf16(rng, (B, g.n_q_heads, d))) * loud)
    k, v = (S.normal_bf16(rng, (B, 2, d)) for _ in range(2))
    pos = rng.integers(0, 131072, B)
    got = _run(g, pool, held, q, k, v, pos, True)
    for b, n in enumerate(held):
        kr = _round_key(_rotate(g, _f64(k[b])[None], [pos[b]]))[0]
        pool.put(0, b, n, 0, kr[:, None])
        pool.put(0, b, n, 1, _f64(v[b])[:, None])
        K, V = (Q.held(pool.codes[i][0], pool.scales[i][0], 32, pool.table[b], n + 1) for i in (0, 1))
        qr = _rotate(g, _f64(q[b])[None], [pos[b]])[0]
        ref = Q.attend(qr, K, V)
        err = np.linalg.norm(got[b] - ref, axis=-1)
        assert (err <= mean_square_bar(qr, K, V, ref)).all(), (err / mean_square_bar(qr, K, V, ref)).max()


@pytest.mark.gpu
@pytest.mark.parametrize("d,group,page", [(128, 4, 64), (64, 8, 16)])
def test_answers_of_a_request_batch_in_the_mean_square(d, group, page):
    from compressed_composable_kv_gb300 import synth as S
    from gpu_util import to_bits
    from test_gpu_pages8 import _f64, _rotate
    from test_gpu_pages8_path import Requests
    r = Requests(S.Geometry(2, 2 * group, 2, d, 5.0e5), page)
    for t in range(r.steps):
        outs = r.outs()
        r.step(t, outs)
        torch.cuda.synchronize()
        want = r.oracle_step(t)
        for l in range(2):
            for b, n0 in enumerate(r.rows):
                K, V = (Q.held(r.codes[i][l], r.scales[i][l], page, r.table[b], n0 + t + 1) for i in (0, 1))
                qr = _rotate(r.g, _f64(to_bits(r.dev["qd_pre"][t, l, b]))[None], [r.rb.l_tot[b] + r.rb.q_len + t])[0]
                ref = want[l][b][0]
                err = np.linalg.norm(outs[l][b].double().cpu().numpy() - ref, axis=-1)
                assert (err <= mean_square_bar(qr, K, V, ref)).all(), f"step {t} layer {l} sequence {b}"
    r.sc.close()
