"""The 8-bit paged cache (filling it, appending to it, attending over it) and
the log probabilities of tokens: the cases that are timed, their plain form
in elementary torch operations, and their values in 64 bits.

A page holds `page` tokens of one layer: for each kv head `page` rows of
head_dim e4m3 codes and one power-of-two scale; a held value is code * scale.
"""
import math
from types import SimpleNamespace

import torch

own = False

E4M3_MAX = 448.0
MIN_EXPONENT = -120

# Head layouts: the repository's Llama-3.1-8B, Qwen3-14B and tiny geometries, and generic ones of the same kind.
GEOMETRIES = {
    "llama8b": (32, 8, 128, 5.0e5),
    "qwen14b": (40, 8, 128, 1.0e6),
    "tiny": (4, 2, 64, 1.0e4),
    "mha": (8, 8, 64, 1.0e4),
    "pairs": (16, 8, 128, 1.0e4),
    "wide": (64, 8, 128, 5.0e5),
}
VOCABS = (128256, 32000, 50257, 151936)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a few short composed caches of the tiny geometry, the smallest fill
        dict(name="fill tiny ragged", op="fill", geom="tiny", layers=1, lens="113,7,1,400", page=16),
        # every layer of one 8000-slot request of the Llama geometry, once per request after its question's prefill
        dict(name="fill 32x8000", op="fill", geom="llama8b", layers=32, lens="8000", page=64),
        # one answer token of a batch of 16: the smallest append, latency counts
        dict(name="append 16x1", op="append", geom="llama8b", batch=16, t_len=1, lo=500, hi=8000, page=64, ragged=False),
        # the questions of 8 requests, padded to 128 tokens, onto caches that end inside a page
        dict(name="append 8x128 ragged", op="append", geom="qwen14b", batch=8, t_len=128, lo=0, hi=8000, page=32, ragged=True),
        # one long uncompressed document appended at once to an empty cache
        dict(name="append 1x4000", op="append", geom="llama8b", batch=1, t_len=4000, lo=0, hi=0, page=128, ragged=False),
        # a small batch of short chats of the tiny head width
        dict(name="attend 16 short", op="attend", geom="tiny", batch=16, lo=1, hi=300, page=16, sharp=1.0),
        # one 8000-slot request, where latency counts
        dict(name="attend 1x8000", op="attend", geom="llama8b", batch=1, lo=8000, hi=8000, page=64, sharp=1.0),
        # 16 requests of different lengths
        dict(name="attend 16 ragged", op="attend", geom="llama8b", batch=16, lo=1000, hi=8000, page=32, sharp=4.0),
        # 8 Qwen3-14B requests of 8000 slots, 5 query heads to a kv head, the smallest page
        dict(name="attend 8x8000 g5", op="attend", geom="qwen14b", batch=8, lo=8000, hi=8000, page=16, sharp=1.0),
        # 4 requests of 128k original tokens at k = 4: the largest
        dict(name="attend 4x32768", op="attend", geom="llama8b", batch=4, lo=32768, hi=32768, page=128, sharp=1.0),
        # the next-token logits of a decode step of 4 requests
        dict(name="logprobs 4 rows", op="logprobs", rows=4, vocab=128256, dtype="bfloat16", top_k=5, masked=False),
        # the logits of a 256-token prompt in 32 bits, an odd vocabulary, some of it masked out
        dict(name="logprobs 256 rows f32", op="logprobs", rows=256, vocab=50257, dtype="float32", top_k=20, masked=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["fill", "append", "attend", "attend", "logprobs"])
    page = rng.choice([16, 32, 64, 128])
    geom = rng.choice(sorted(GEOMETRIES))
    if op == "fill":
        n = rng.randint(1, 16)
        lens = [_log_int(rng, 1, 4000) for _ in range(n)]
        layers = max(1, min(rng.randint(1, 32), 120000 // sum(lens)))
        return dict(op=op, geom=geom, layers=layers, lens=",".join(map(str, lens)), page=page)
    if op == "append":
        batch = _log_int(rng, 1, 64)
        return dict(op=op, geom=geom, batch=batch, t_len=_log_int(rng, 1, max(1, 4000 // batch)), lo=0, hi=_log_int(rng, 1, 4000), page=page,
                    ragged=rng.random() < 0.5)
    if op == "attend":
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, 100000 // batch)
        return dict(op=op, geom=geom, batch=batch, lo=rng.randint(0, hi), hi=hi, page=page, sharp=rng.choice([1.0, 4.0]))
    vocab = rng.choice(VOCABS + (_log_int(rng, 1, 200000),))
    return dict(op=op, rows=_log_int(rng, 1, max(1, min(512, 20000000 // vocab))), vocab=vocab, dtype=rng.choice(["bfloat16", "float32"]),
                top_k=min(vocab, rng.choice([0, 1, 5, 8, 20, 32])), masked=rng.random() < 0.5)


def work(case):
    if case["op"] == "logprobs":
        n = case["rows"] * case["vocab"]
        size = 2 if case["dtype"] == "bfloat16" else 4
        return {"bytes": n * size + case["rows"] * (12 + 8 * case["top_k"]), "flops": 5 * n}
    hq, hkv, d, _ = GEOMETRIES[case["geom"]]
    row = 2 * hkv * d  # elements of K and V of one token
    if case["op"] == "fill":
        lens = [int(x) for x in case["lens"].split(",")]
        pages = sum(-(-n // case["page"]) for n in lens)
        return {"bytes": case["layers"] * (sum(lens) * row * 3 + pages * hkv * 8), "flops": case["layers"] * sum(lens) * row * 3}
    lens = _lengths(case)
    if case["op"] == "append":
        tokens = sum(_new_lengths(case))
        return {"bytes": tokens * (row * 3 + d // 2 * 16), "flops": tokens * row * 6}
    keys = sum(n + 1 for n in lens)
    pages = sum(n // case["page"] + 1 for n in lens)
    moved = keys * row + pages * hkv * 8 + len(lens) * (4 * hq * d + 2 * row + d // 2 * 16)
    return {"bytes": moved, "flops": 4 * keys * hq * d}


def _lengths(case):
    """Cached tokens of each sequence: between lo and hi, both of them among the lengths, the same for every seed."""
    b, lo, hi = case["batch"], case["lo"], case["hi"]
    return [hi if i == 0 else lo if i == 1 else lo + (i * 2654435761 % 4294967296) * (hi - lo + 1) // 4294967296 for i in range(b)]


def _new_lengths(case):
    """New tokens of each sequence; a ragged batch has a full one, an empty one and others between."""
    t = case["t_len"]
    if not case["ragged"]:
        return [t] * case["batch"]
    return [t if i == 0 else 0 if i == 1 else 1 + (i * 2246822519 % 4294967296) * t // 4294967296 for i in range(case["batch"])]


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*size):
        return torch.randn(size, generator=gen, device="cuda")

    if case["op"] == "logprobs":
        rows, vocab, k = case["rows"], case["vocab"], case["top_k"]
        x = normal(rows, vocab) * 2.5
        x[:, : max(1, vocab // 1000)] += 4.0  # a few likely tokens
        if case["masked"]:  # tokens that the caller rules out
            x[torch.rand(rows, vocab, generator=gen, device="cuda") < 0.2] = -math.inf
        tokens = torch.randint(0, vocab, (rows,), generator=gen, device="cuda", dtype=torch.int32)
        tokens[rows // 2 + 1 :: 7] = -1  # rows that have no given token
        return dict(case=case, logits=x.to(getattr(torch, case["dtype"])), tokens=tokens, logprob=torch.zeros(rows, device="cuda"), entropy=torch.zeros(rows, device="cuda"),
                    top_ids=torch.zeros(rows, k, dtype=torch.int32, device="cuda"), top_logprobs=torch.zeros(rows, k, device="cuda"))

    hq, hkv, d, theta = GEOMETRIES[case["geom"]]
    page = case["page"]
    layers = case.get("layers", 1)
    geom = SimpleNamespace(n_layers=layers, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, rope_theta=theta)
    if case["op"] == "fill":
        lens = held = [int(x) for x in case["lens"].split(",")]
        total = lens
    else:
        held = _lengths(case)
        new = _new_lengths(case) if case["op"] == "append" else [1] * case["batch"]
        total = [h + n for h, n in zip(held, new)]
    counts = [-(-t // page) for t in total]
    n_pages = sum(counts) + 3
    most = max(counts) + 1
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    at = torch.arange(most, device="cuda")
    start = torch.tensor([sum(counts[:i]) for i in range(len(counts))], device="cuda")[:, None]
    table = torch.where(at < torch.tensor(counts, device="cuda")[:, None], order[(start + at).clamp(max=n_pages - 1)], -1).to(torch.int32).contiguous()
    # keys have a few channels that stand out, values do not; all pages hold something, as a pool in use does
    loud = 1.0 + 5.0 * (torch.rand(hkv, 1, d, generator=gen, device="cuda") < 0.03)
    s = dict(case=case, geom=geom, page_table=table)
    for name, factor in (("k", loud), ("v", torch.ones_like(loud))):
        codes = torch.empty(layers, n_pages, hkv, page, d, dtype=torch.float8_e4m3fn, device="cuda")
        scales = torch.empty(layers, n_pages, hkv, device="cuda")
        for l in range(layers):
            codes[l], scales[l] = _quantise((normal(n_pages, hkv, page, d) * factor).to(torch.bfloat16).float())
        s[name + "8"], s[name + "_scale"] = codes, scales
    if case["op"] == "fill":
        cap = -(-max(lens) // 32) * 32
        s.update(cap=cap, n_rows=lens, k_caches=[(normal(layers, hkv, cap, d) * loud).to(torch.bfloat16) for _ in lens],
                 v_caches=[normal(layers, hkv, cap, d).to(torch.bfloat16) for _ in lens])
        return s
    t_len = case.get("t_len", 1)
    batch = case["batch"]
    # RoPE rows as the framework's table holds them: cos and sin as pairs of 32-bit numbers, at positions up to 128k
    pos = torch.randint(0, 131072, (batch,), generator=gen, device="cuda")[:, None] + torch.arange(t_len, device="cuda")
    angle = pos.reshape(-1, 1).double() * theta ** (-2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    parts = [p for f in (angle.cos(), angle.sin()) for p in (f.float(), (f - f.float().double()).float())]
    s.update(rope_table=torch.stack(parts, -1).contiguous(), rope_row=torch.arange(batch, device="cuda", dtype=torch.int32) * t_len,
             n_cached=torch.tensor(held, device="cuda", dtype=torch.int32), max_keys=max(total), t_len=t_len)
    s["k_new"] = (normal(batch, t_len, hkv, d) * loud.reshape(1, 1, hkv, d)).to(torch.bfloat16)
    s["v_new"] = normal(batch, t_len, hkv, d).to(torch.bfloat16)
    if case["op"] == "append":
        s["n_new"] = torch.tensor(new, device="cuda", dtype=torch.int32) if case["ragged"] else None
    else:
        s["k_new"], s["v_new"] = s["k_new"][:, 0].contiguous(), s["v_new"][:, 0].contiguous()
        s["q"] = (normal(batch, hq, d) * case["sharp"] / 2.0).to(torch.bfloat16)
        s["out"] = torch.zeros(batch, hq, d, dtype=torch.bfloat16, device="cuda")
        s["workspace"] = torch.zeros(8 << 20, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        import compressed_composable_kv_gb300 as P
        if op == "logprobs":
            P.c2kv_token_logprobs(state["logits"], state["tokens"], state["top_ids"].shape[1], state["logprob"], state["entropy"], state["top_ids"], state["top_logprobs"])
        elif op == "fill":
            P.c2kv_pages8_fill(state["geom"], 0, state["geom"].n_layers, state["k_caches"], state["v_caches"], state["cap"], state["n_rows"], state["k8"], state["v8"],
                               state["k_scale"], state["v_scale"], state["page_table"])
        elif op == "append":
            P.c2kv_pages8_append(state["geom"], 0, state["k8"], state["v8"], state["k_scale"], state["v_scale"], state["page_table"], state["n_cached"], state["k_new"],
                                 state["v_new"], state["rope_table"], state["rope_row"], state["n_new"])
        else:
            P.c2kv_attend_pages8(state["geom"], 0, state["k8"], state["v8"], state["k_scale"], state["v_scale"], state["page_table"], state["n_cached"], state["max_keys"],
                                 state["q"], state["k_new"], state["v_new"], state["rope_table"], state["rope_row"], state["out"], state["workspace"])
    elif op == "logprobs":
        _plain_logprobs(state)
    elif op == "fill":
        _plain_fill(state)
    else:
        one = op == "attend"
        new = state["n_new"] if not one and state["n_new"] is not None else torch.full_like(state["n_cached"], state["t_len"])
        _plain_append(state, state["k_new"][:, None] if one else state["k_new"], state["v_new"][:, None] if one else state["v_new"], new)
        if one:
            state["out"].copy_(_plain_attend(state))
    if op == "logprobs":
        return {name: state[name] for name in ("logprob", "entropy", "top_ids", "top_logprobs")}
    held = {name: state[name] for name in ("k8", "v8", "k_scale", "v_scale")}
    return held if op != "attend" else dict(held, out=state["out"])


# ------------------------------------------------------------------ the plain form

def _exponent(a):
    """The smallest e with a <= 448 * 2^e = 1.75 * 2^(8 + e), at least MIN_EXPONENT."""
    m, x = torch.frexp(a)
    return torch.where(2.0 * m <= 1.75, x - 9, x - 8).clamp(min=MIN_EXPONENT).where(a > 0, torch.full_like(x, MIN_EXPONENT))


def _times_power(x, e):
    return (x.double() * torch.exp2(e.double())).float()


def _quantise(x):
    """Codes and scales of [..., page, d] values, one scale for the last two axes."""
    fine = x.isfinite()
    e = _exponent(torch.where(fine, x.abs(), 0.0).amax((-2, -1)))
    y = _times_power(x, -e[..., None, None])
    return torch.where(fine, y, math.nan).to(torch.float8_e4m3fn), torch.exp2(e.double()).float()


def _plain_fill(s):
    page, table = s["case"]["page"], s["page_table"].long()
    lens = torch.tensor(s["n_rows"], device=table.device)
    rows = torch.arange(table.shape[1] * page, device=table.device).reshape(1, -1, page)
    valid = rows < lens[:, None, None]  # [batch][page of the sequence][row]
    hit = valid[:, :, 0]
    pad = table.shape[1] * page - s["cap"]
    for caches, codes, scales in ((s["k_caches"], s["k8"], s["k_scale"]), (s["v_caches"], s["v8"], s["v_scale"])):
        for l in range(codes.shape[0]):
            x = torch.stack([c[l] for c in caches]).float()  # [batch][head][cap][d]
            x = torch.nn.functional.pad(x, (0, 0, 0, max(0, pad)))[:, :, : table.shape[1] * page]
            x = x.reshape(len(caches), codes.shape[2], -1, page, codes.shape[4]).transpose(1, 2)[hit]  # [pages][head][page][d]
            keep = valid[hit][:, None, :, None]
            new, scale = _quantise(torch.where(keep, x, 0.0))
            at = table[hit]
            raw = codes[l].view(torch.uint8)
            raw[at] = torch.where(keep, new.view(torch.uint8), raw[at])
            scales[l, at] = scale


def _rope(s, row):
    """cos and sin, in 64 bits, of the given rows of the table."""
    t = s["rope_table"][row].double()
    return t[..., 0] + t[..., 1], t[..., 2] + t[..., 3]


def _rotate(x, cos, sin):
    a, b = x.double().chunk(2, -1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _plain_append(s, k_new, v_new, n_new):
    page, table, n = s["case"]["page"], s["page_table"].long(), s["n_cached"].long()
    batch, t_len = k_new.shape[:2]
    i = torch.arange(t_len, device=n.device)
    cos, sin = _rope(s, s["rope_row"].long()[:, None] + i)
    k_new = _rotate(k_new, cos[:, :, None], sin[:, :, None]).float().to(torch.bfloat16)
    touched = (page - 1 + t_len - 1) // page + 1
    first = n // page
    rows = (first[:, None] * page + torch.arange(touched * page, device=n.device)).reshape(batch, touched, page)
    token = rows - n[:, None, None]
    is_new, is_old = (token >= 0) & (token < n_new.long()[:, None, None]), token < 0
    hit = is_new.any(-1)
    at = table.gather(1, (first[:, None] + torch.arange(touched, device=n.device)).clamp(max=table.shape[1] - 1))[hit]
    has_old = is_old[hit].any(-1)[:, None]
    fresh, old = is_new[hit][:, None, :, None], is_old[hit][:, None, :, None]
    pick = token.clamp(0, t_len - 1)
    which = torch.arange(batch, device=n.device)[:, None, None].expand_as(pick)
    for x, codes, scales in ((k_new, s["k8"][0], s["k_scale"][0]), (v_new, s["v8"][0], s["v_scale"][0])):
        x = torch.where(fresh, x[which[hit], pick[hit]].transpose(1, 2).float(), 0.0)  # [pages][head][page][d]
        raw = codes.view(torch.uint8)
        was, before = raw[at], scales[at]
        fine = x.isfinite()
        e = _exponent(torch.where(fine, x.abs(), 0.0).amax((-2, -1)))
        e_old = torch.frexp(before)[1] - 1
        e = torch.where(has_old, torch.maximum(e, e_old), e)
        coarser = _times_power(was.view(torch.float8_e4m3fn).float(), (e_old - e).clamp(max=0)[..., None, None]).to(torch.float8_e4m3fn)
        new = torch.where(fine, _times_power(x, -e[..., None, None]), math.nan).to(torch.float8_e4m3fn)
        raw[at] = torch.where(fresh, new.view(torch.uint8), torch.where(old, coarser.view(torch.uint8), was))
        scales[at] = torch.exp2(e.double()).float()


def _plain_attend(s):
    table, n = s["page_table"].long().clamp(min=0), s["n_cached"].long()
    batch, hq, d = s["q"].shape
    cos, sin = _rope(s, s["rope_row"].long())
    q = _rotate(s["q"], cos[:, None], sin[:, None]).float()

    def values(codes, scales):
        x = codes[0].view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * scales[0][table][..., None, None]
        return x.transpose(1, 2).reshape(batch, x.shape[2], -1, d)  # [batch][kv head][key][d]

    k = values(s["k8"], s["k_scale"])
    score = q.reshape(batch, k.shape[1], -1, d) @ k.transpose(2, 3) / math.sqrt(d)
    seen = torch.arange(k.shape[2], device=n.device) <= n[:, None, None, None]
    score = torch.where(seen, score, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    v = torch.where(seen.reshape(batch, 1, -1, 1), values(s["v8"], s["v_scale"]), 0.0)
    return (p @ v / p.sum(-1, keepdim=True)).reshape(batch, hq, d).to(torch.bfloat16)


def _plain_logprobs(s):
    x = s["logits"].float()
    rows, vocab = x.shape
    top = x.amax(-1, keepdim=True)
    y = x - top
    p = torch.exp(y)
    total = p.sum(-1, keepdim=True)
    lse = torch.log(total)
    given = s["tokens"].long()
    lp = y.gather(1, given.clamp(min=0)[:, None]) - lse
    s["logprob"].copy_(torch.where(given < 0, 0.0, lp[:, 0]))
    s["entropy"].copy_((lse - torch.where(p > 0, p * y, 0.0).sum(-1, keepdim=True) / total)[:, 0])
    k = s["top_ids"].shape[1]
    if k:
        bits = x.view(torch.int32).long()  # an order of whole numbers: larger value first, then the lower index
        bits = torch.where(bits < 0, -(bits + (1 << 31)) , bits)
        key = bits * (1 << 20) + (vocab - 1 - torch.arange(vocab, device=x.device))
        ids = vocab - 1 - (torch.topk(key, k, dim=-1).values & ((1 << 20) - 1))
        s["top_ids"].copy_(ids)
        s["top_logprobs"].copy_(y.gather(1, ids) - lse)


# ------------------------------------------------------------------ 64 bits, written apart from the above

def _e4m3(x):
    """x, in 64 bits, on the grid of e4m3: 3 bits after the leading one, down to steps of 2^-9; halves go to even."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (x / step).round() * step


def _scale_of(largest):
    """2^e with 224 < largest / 2^e <= 448."""
    e = torch.ceil(torch.log2(largest.clamp(min=1e-300) / E4M3_MAX))
    e = torch.where(largest > E4M3_MAX * torch.exp2(e), e + 1, e)
    e = torch.where(largest <= E4M3_MAX * torch.exp2(e - 1), e - 1, e)
    return torch.exp2(e.clamp(min=MIN_EXPONENT))


def _exact_put(codes, scales, l, ids, page, first, x):
    """Rows first, first + 1, ... of a sequence get x [head][rows][d]."""
    done = 0
    while done < x.shape[1]:
        row = (first + done) % page
        take = min(page - row, x.shape[1] - done)
        pid = int(ids[(first + done) // page])
        part = x[:, done : done + take]
        scale = _scale_of(part.abs().amax((1, 2)))
        if row:
            scale = torch.maximum(scale, scales[l, pid])
            codes[l, pid, :, :row] = _e4m3(codes[l, pid, :, :row] * (scales[l, pid] / scale)[:, None, None])
        codes[l, pid, :, row : row + take] = _e4m3(part / scale[:, None, None])
        scales[l, pid] = scale
        done += take


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        x = s["logits"].double()
        logp = x - torch.logsumexp(x, -1, keepdim=True)
        given = s["tokens"].long()
        value, at = torch.sort(x, dim=-1, descending=True, stable=True)
        k = case["top_k"]
        rows = torch.arange(len(given), device=x.device)
        return {"logprob": torch.where(given >= 0, logp[rows, given.clamp(min=0)], 0.0), "entropy": torch.special.entr(logp.exp()).sum(-1),
                "top_ids": at[:, :k].to(torch.int32), "top_logprobs": logp.gather(1, at[:, :k])}
    page = case["page"]
    got = {name: s[name].double() for name in ("k8", "v8", "k_scale", "v_scale")}
    if case["op"] == "fill":
        if s["geom"].n_layers * sum(-(-n // page) for n in s["n_rows"]) > 20000:
            return None
        for b, n in enumerate(s["n_rows"]):
            ids = s["page_table"][b].tolist()
            for l in range(s["geom"].n_layers):
                for name in "kv":
                    _exact_put(got[name + "8"], got[name + "_scale"], l, ids, page, 0, s[name + "_caches"][b][l, :, :n].double())
        return got
    one = case["op"] == "attend"
    held = s["n_cached"].tolist()
    news = [1] * len(held) if one else _new_lengths(case)
    tables = s["page_table"].tolist()
    hkv, d = s["geom"].n_kv_heads, s["geom"].head_dim
    out = []
    for b, (n, t) in enumerate(zip(held, news)):
        k_new, v_new = (s[name][b].reshape(-1, hkv, d)[:t].double() for name in ("k_new", "v_new"))
        rope = s["rope_table"][int(s["rope_row"][b]) :][:max(t, 1)].double()
        turn = torch.complex(rope[..., 0] + rope[..., 1], rope[..., 2] + rope[..., 3])[:, None]
        z = torch.complex(k_new[..., : d // 2], k_new[..., d // 2 :]) * turn[:t]
        k_new = torch.cat((z.real, z.imag), -1).to(torch.bfloat16).double()
        _exact_put(got["k8"], got["k_scale"], 0, tables[b], page, n, k_new.transpose(0, 1))
        _exact_put(got["v8"], got["v_scale"], 0, tables[b], page, n, v_new.transpose(0, 1))
        if one:
            ids = torch.tensor(tables[b][: n // page + 1], device="cuda")
            k, v = ((got[name + "8"][0, ids] * got[name + "_scale"][0, ids][..., None, None]).transpose(0, 1).reshape(hkv, -1, d)[:, : n + 1] for name in "kv")
            q = s["q"][b].double().reshape(hkv, -1, d)
            z = torch.complex(q[..., : d // 2], q[..., d // 2 :]) * turn[0]
            p = torch.softmax(torch.cat((z.real, z.imag), -1) @ k.transpose(1, 2) * d ** -0.5, -1)
            out.append((p @ v).reshape(-1, d))
    return dict(got, out=torch.stack(out)) if one else got
