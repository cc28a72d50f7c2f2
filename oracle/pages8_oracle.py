"""Plain fp64 CPU oracle of the 8-bit paged cache and of the token log
probabilities.  Test infrastructure only: no product code imports it.

A page of one (layer, kv head) is `page` rows of e4m3 codes under one scale
2^e; values here are numpy float64, codes are uint8 bit patterns.
"""
import numpy as np

MIN_EXPONENT = -120


def _all_e4m3() -> np.ndarray:
    """Value of every code 0..255, by the format's definition: sign, 4 exponent
    bits with bias 7, 3 mantissa bits, no infinity, 0x7F and 0xFF are NaN."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        out[c] = np.nan if (c & 127) == 127 else (-v if s else v)
    return out


E4M3 = _all_e4m3()
_POS = E4M3[:127]   # 0 .. 448, ascending


def e4m3_values(codes: np.ndarray) -> np.ndarray:
    return E4M3[codes]


def e4m3_codes(x: np.ndarray) -> np.ndarray:
    """|x| <= 448 or NaN to the nearest code, halves to the even one."""
    a = np.abs(x)
    a = np.where(np.isnan(a), 0.0, a)
    assert a.max(initial=0.0) <= 448.0
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 1, 126)
    lo = hi - 1
    below, above = a - _POS[lo], _POS[hi] - a
    c = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    c = c | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(0x7F), c)


def scale_exponent(x: np.ndarray) -> int:
    """The smallest e >= MIN_EXPONENT with every finite |x| <= 448 * 2^e."""
    fin = np.abs(x[np.isfinite(x)])
    a = fin.max(initial=0.0)
    e = MIN_EXPONENT
    while a > 448.0 * 2.0 ** e:
        e += 1
    return e


def put(codes: np.ndarray, scales: np.ndarray, page: int, table, first: int, x: np.ndarray) -> None:
    """Rows first, first + 1, ... of a sequence get x [kv head][rows][d], in
    place in codes [n_pages][kv head][page][d] and scales [n_pages][kv head]."""
    r = 0
    while r < x.shape[1]:
        at = (first + r) % page
        n = min(page - at, x.shape[1] - r)
        pid = table[(first + r) // page]
        for h in range(x.shape[0]):
            part = x[h, r:r + n].copy()
            e = scale_exponent(part)
            if at:
                e_old = int(np.log2(scales[pid, h]))
                if e > e_old:
                    old = e4m3_values(codes[pid, h, :at]) * 2.0 ** (e_old - e)
                    codes[pid, h, :at] = e4m3_codes(old)
                e = max(e, e_old)
            part[~np.isfinite(part)] = np.nan
            codes[pid, h, at:at + n] = e4m3_codes(part * 2.0 ** -e)
            scales[pid, h] = 2.0 ** e
        r += n


def held(codes: np.ndarray, scales: np.ndarray, page: int, table, n: int) -> np.ndarray:
    """The n held rows of a sequence, [kv head][n][d]."""
    pids = np.asarray(table)[: -(-n // page)].astype(int)
    x = e4m3_values(codes[pids]) * scales[pids].astype(np.float64)[:, :, None, None]
    return x.transpose(1, 0, 2, 3).reshape(codes.shape[1], -1, codes.shape[3])[:, :n]


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray) -> np.ndarray:
    """q [q heads][d] rotated; k, v [kv head][n][d] held values; 0 for n = 0."""
    hq, d = q.shape
    group = hq // k.shape[0]
    out = np.zeros((hq, d))
    if k.shape[1] == 0:
        return out
    for h in range(hq):
        s = k[h // group] @ q[h] / np.sqrt(d)
        p = np.exp(s - s.max())
        out[h] = p @ v[h // group] / p.sum()
    return out


def token_logprobs(x: np.ndarray, tokens, top_k: int):
    """(logprob, entropy, top_ids, top_logprobs) of logits x [rows][vocab]."""
    rows, vocab = x.shape
    lp, ent = np.zeros(rows), np.zeros(rows)
    ids, tops = np.zeros((rows, top_k), np.int32), np.zeros((rows, top_k))
    for r in range(rows):
        # larger first (NaN above all), then the lower index
        order = np.lexsort((np.arange(vocab), -np.where(np.isnan(x[r]), 0.0, x[r]), ~np.isnan(x[r])))
        if np.isnan(x[r]).any() or np.isposinf(x[r]).any():
            all_lp, ent[r] = np.full(vocab, np.nan), np.nan
        elif np.isneginf(x[r]).all():
            all_lp, ent[r] = np.full(vocab, -np.inf), 0.0
        else:
            y = x[r] - x[r].max()
            all_lp = y - np.log(np.exp(y).sum())
            p = np.exp(all_lp)
            ent[r] = -(p[p > 0] * all_lp[p > 0]).sum()
        ids[r], tops[r] = order[:top_k], all_lp[order[:top_k]]
        if tokens is not None and tokens[r] >= 0:
            lp[r] = all_lp[tokens[r]]
    return lp, ent, ids, tops
