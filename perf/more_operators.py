"""Attention of a chunk of new tokens over the 8-bit paged cache, and the pages
of a cache among its sequences (forking, freeing and reserving, compacting): the
cases that are timed, their plain form in elementary torch operations, and their
values in 64 bits.

A page holds `page` tokens of one layer: for each kv head `page` rows of
head_dim e4m3 codes and one power-of-two scale; a held value is code * scale.  A
row of the page table names a sequence's pages, negative behind them; refs counts
how many sequences hold a page, 0 where it is free.
"""
import math
import random
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
MOST_SCORES = 32 * 4 * 512 * 33280  # of the largest listed chunk
MOST_POOL = 1 << 30                 # bytes of K and V codes of a drawn pool
MOST_COPIED = 140 << 20             # bytes that a drawn fork copies


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a few drafted tokens of short chats checked at once: the smallest chunk, latency counts
        dict(name="chunk 8x4 tiny", op="chunk", geom="tiny", batch=8, t_len=4, lo=1, hi=300, page=16, ragged=False, sharp=1.0),
        # up to 5 drafted tokens for each of 16 requests of different lengths: the bytes of the pages count
        dict(name="chunk 16x5 drafts", op="chunk", geom="llama8b", batch=16, t_len=5, lo=1000, hi=8000, page=64, ragged=True, sharp=4.0),
        # a second question on one 8000-slot request
        dict(name="chunk 1x64 over 8000", op="chunk", geom="llama8b", batch=1, t_len=64, lo=8000, hi=8000, page=64, ragged=False, sharp=1.0),
        # second questions of 8 Qwen3-14B requests, padded to 128 tokens, 5 query heads to a kv head
        dict(name="chunk 8x128 g5", op="chunk", geom="qwen14b", batch=8, t_len=128, lo=7000, hi=8000, page=32, ragged=True, sharp=1.0),
        # heads of 64 without groups, odd lengths, the smallest page
        dict(name="chunk 3x333 d64", op="chunk", geom="mha", batch=3, t_len=333, lo=100, hi=4999, page=16, ragged=True, sharp=4.0),
        # an uncompressed document of 4000 tokens taken in at once into an empty cache
        dict(name="chunk 1x4000", op="chunk", geom="llama8b", batch=1, t_len=4000, lo=0, hi=0, page=128, ragged=False, sharp=1.0),
        # a piece of 512 tokens onto each of 4 requests of 128k original tokens at k = 4: the largest
        dict(name="chunk 4x512 over 32768", op="chunk", geom="llama8b", batch=4, t_len=512, lo=32768, hi=32768, page=64, ragged=False, sharp=1.0),
        # three short chats forked into seven: the smallest fork
        dict(name="fork 3 to 7 tiny", op="fork", geom="tiny", layers=2, batch=3, out=7, lo=5, hi=130, page=16, room=1, beam=0),
        # 8 answers to each of 4 prefilled requests, all layers, room for 100 tokens each
        dict(name="fork 4 to 32", op="fork", geom="llama8b", layers=32, batch=4, out=32, lo=1500, hi=1999, page=128, room=100, beam=0),
        # one step of a search with 8 beams for each of 8 requests: beams are dropped, go on and split
        dict(name="fork 8x8 beams", op="fork", geom="pairs", layers=8, batch=64, out=64, lo=500, hi=2000, page=16, room=1, beam=8),
        # a small pool after some chats have ended
        dict(name="compact tiny", op="compact", geom="tiny", layers=2, batch=5, lo=10, hi=200, page=16, pages=97, shared=2),
        # half of a pool in use after many requests have come and gone
        dict(name="compact 512 pages", op="compact", geom="llama8b", layers=16, batch=14, lo=1000, hi=2200, page=64, pages=512, shared=4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "fork", "compact"])
    page = rng.choice([16, 32, 64, 128])
    geom = rng.choice(sorted(GEOMETRIES))
    hq, hkv, d, _ = GEOMETRIES[geom]
    if op == "chunk":
        batch = _log_int(rng, 1, 64)
        t_len = _log_int(rng, 1, max(1, 4000 // batch))
        most = min(100000 // batch, MOST_SCORES // (hq * batch * t_len) - t_len)
        hi = _log_int(rng, 1, max(1, most)) if rng.random() < 0.9 else 0
        return dict(op=op, geom=geom, batch=batch, t_len=t_len, lo=rng.randint(0, hi), hi=hi, page=page, ragged=rng.random() < 0.5,
                    sharp=rng.choice([1.0, 4.0]))
    layers = _log_int(rng, 1, 32)
    page_bytes = 2 * layers * hkv * page * d
    batch = _log_int(rng, 1, 64)
    pages = max(2 * batch, MOST_POOL // page_bytes)  # that the sequences may hold
    hi = max(1, min(_log_int(rng, 1, 8000), (pages // (2 * batch) - 1) * page + rng.randint(0, page - 1)))
    lo = rng.randint(0, hi)
    if op == "compact":
        case = dict(op=op, geom=geom, layers=layers, batch=batch, lo=lo, hi=hi, page=page, pages=0, shared=rng.choice([0, 1, 4]))
        used = _used(case)
        return dict(case, pages=used + rng.randint(0, max(1, min(2 * used, MOST_POOL // page_bytes - used))))
    beam = rng.choice([0, 0, 2, 4, 8])
    out = batch if beam else batch * rng.choice([1, 2, 3, 4])
    room = rng.choice([0, 1, 1, page, 5 * page // 2])
    out = max(1, min(out, MOST_COPIED // page_bytes))
    return dict(op=op, geom=geom, layers=layers, batch=batch, out=out, lo=lo, hi=hi, page=page, room=room, beam=beam)


def work(case):
    hq, hkv, d, _ = GEOMETRIES[case["geom"]]
    page = case["page"]
    row = 2 * hkv * d  # elements of K and V of one token
    if case["op"] == "chunk":
        held, new = _lengths(case), _new_lengths(case)
        tokens = sum(new)
        seen = sum(t * n + t * (t + 1) // 2 for n, t in zip(held, new))
        rows = sum(n + t for n, t in zip(held, new) if t)
        pages = sum(-(-(n + t) // page) for n, t in zip(held, new) if t)
        return {"bytes": rows * row + pages * hkv * 8 + tokens * (4 * hq * d + 2 * row + row + d // 2 * 16), "flops": 4 * seen * hq * d + tokens * row * 6}
    if case["op"] == "compact":
        return {"bytes": 2 * case["layers"] * _moves(case) * (page * row + hkv * 8) + 8 * case["batch"] * _width(case) + 12 * case["pages"], "flops": 0}
    plan = _fork_plan(case)
    moved = sum(2 * case["layers"] * (rows * row + hkv * 8) for rows in plan["copied"])
    return {"bytes": moved + 4 * (case["batch"] + case["out"]) * _width(case) + 8 * _pool_pages(case), "flops": 0}


def _spread(i, n):
    """A whole number in [0, n) that goes with i."""
    return (i * 2654435761 % 4294967296) * n // 4294967296


def _lengths(case):
    """Cached tokens of each sequence: between lo and hi, both of them among the lengths, the same for every seed."""
    lo, hi = case["lo"], case["hi"]
    return [hi if i == 0 else lo if i == 1 else lo + _spread(i, hi - lo + 1) for i in range(case["batch"])]


def _new_lengths(case):
    """New tokens of each sequence; a ragged batch has a full one, an empty one and others between."""
    t = case["t_len"]
    if not case["ragged"]:
        return [t] * case["batch"]
    return [t if i == 0 else 0 if i == 1 else 1 + (i * 2246822519 % 4294967296) * t // 4294967296 for i in range(case["batch"])]


def _layout(case):
    """Pages of each sequence, and how many of the first of them it shares with the first sequence of its group."""
    page, lens = case["page"], _lengths(case)
    group = case.get("beam") or case.get("shared") or 1
    counts = [-(-n // page) for n in lens]
    common = []
    for b, n in enumerate(lens):
        mates = lens[b // group * group : (b // group + 1) * group]
        common.append(min(mates) // page * 3 // 4 if group > 1 and b % group else 0)
    return counts, common


def _used(case):
    counts, common = _layout(case)
    return sum(counts) - sum(common)


def _width(case):
    """Entries of a row of the page table."""
    return -(-(case["hi"] + case.get("room", 0)) // case["page"]) + 2


def _moves(case):
    """Pages in use that lie behind as many pages as are in use."""
    used = _used(case)
    return used * (case["pages"] - used) // max(1, case["pages"])


def _parents(case):
    """The sequence that each place of the new batch goes on with; -1: none."""
    n, beam = case["batch"], case["beam"]
    if not beam:
        return [i % n for i in range(case["out"])]
    r = random.Random(repr(sorted(case.items(), key=str)))
    return [-1 if r.random() < 0.06 else min(n - 1, i // beam * beam + int(beam * r.random() ** 1.7)) for i in range(case["out"])]


def _fork_plan(case):
    """Rows of each copied page, and pages taken."""
    lens, page, parents = _lengths(case), case["page"], _parents(case)
    copied, taken = [], 0
    for i, r in enumerate(parents):
        if r < 0:
            continue
        first = r not in parents[:i]
        keep = -(-lens[r] // page) if first else lens[r] // page
        taken += -(-(lens[r] + case["room"]) // page) - keep if lens[r] + case["room"] > keep * page else 0
        if not first and lens[r] % page:
            copied.append(lens[r] % page)
    return {"copied": copied, "taken": taken}


def _pool_pages(case):
    return _used(case) + _fork_plan(case)["taken"] + 3


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*size):
        return torch.randn(size, generator=gen, device="cuda")

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    hq, hkv, d, theta = GEOMETRIES[case["geom"]]
    page, layers = case["page"], case.get("layers", 1)
    geom = SimpleNamespace(n_layers=layers, n_q_heads=hq, n_kv_heads=hkv, head_dim=d, rope_theta=theta)
    s = dict(case=case, geom=geom)
    held = _lengths(case)
    if case["op"] != "chunk":
        counts, common = _layout(case)
        used = _used(case)
        n_pages = case["pages"] if case["op"] == "compact" else _pool_pages(case)
        r = random.Random(seed)
        if case["op"] == "compact":
            ids = r.sample(range(used, n_pages), _moves(case)) + r.sample(range(used), used - _moves(case))
            r.shuffle(ids)
        else:
            ids = r.sample(range(n_pages), used)
        table, refs, width = [], [0] * n_pages, _width(case)
        group = case.get("beam") or case.get("shared") or 1
        for b, (c, share) in enumerate(zip(counts, common)):
            row = table[b // group * group][:share] if share else []
            row = row + [ids.pop() for _ in range(c - share)]
            for i in row:
                refs[i] += 1
            table.append(row + [-1] * (width - c))
        s.update(page_table=ints(table), refs=ints(refs), refs_out=torch.zeros(n_pages, dtype=torch.int32, device="cuda"),
                 workspace=torch.zeros(16 << 20, dtype=torch.uint8, device="cuda"))
        if case["op"] == "compact":
            s.update(page_table_out=torch.zeros_like(s["page_table"]), moved_out=torch.zeros_like(s["refs"]))
        else:
            s.update(n_cached=ints(held), parent=ints(_parents(case)), n_cached_out=torch.zeros(case["out"], dtype=torch.int32, device="cuda"),
                     page_table_out=torch.zeros(case["out"], width, dtype=torch.int32, device="cuda"))
        for name in "kv":
            codes = torch.empty(layers, n_pages, hkv, page, d, dtype=torch.float8_e4m3fn, device="cuda")
            for l in range(layers):
                codes[l] = (normal(n_pages, hkv, page, d) * 80.0).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            s[name + "8"] = codes
            s[name + "_scale"] = torch.exp2(torch.randint(-8, -4, (layers, n_pages, hkv), generator=gen, device="cuda").float())
        return s
    new = _new_lengths(case)
    batch, t_len = case["batch"], case["t_len"]
    total = [h + t for h, t in zip(held, new)]
    counts = [-(-t // page) for t in total]
    n_pages = sum(counts) + 3
    most = max(counts + [-(-t_len // page)]) + 1
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    at = torch.arange(most, device="cuda")
    start = torch.tensor([sum(counts[:i]) for i in range(len(counts))], device="cuda")[:, None]
    s["page_table"] = torch.where(at < torch.tensor(counts, device="cuda")[:, None], order[(start + at).clamp(max=n_pages - 1)], -1).to(torch.int32).contiguous()
    # keys have a few channels that stand out, values do not; all pages hold something, as a pool in use does
    loud = 1.0 + 5.0 * (torch.rand(hkv, 1, d, generator=gen, device="cuda") < 0.03)
    for name, factor in (("k", loud), ("v", torch.ones_like(loud))):
        codes, scales = _quantise((normal(1, n_pages, hkv, page, d) * factor).to(torch.bfloat16).float())
        s[name + "8"], s[name + "_scale"] = codes, scales
    # RoPE rows as the framework's table holds them: cos and sin as pairs of 32-bit numbers, at positions up to 128k
    pos = torch.randint(0, 131072, (batch,), generator=gen, device="cuda")[:, None] + torch.arange(t_len, device="cuda")
    angle = pos.reshape(-1, 1).double() * theta ** (-2.0 * torch.arange(d // 2, device="cuda", dtype=torch.float64) / d)
    parts = [p for f in (angle.cos(), angle.sin()) for p in (f.float(), (f - f.float().double()).float())]
    s.update(rope_table=torch.stack(parts, -1).contiguous(), rope_row=torch.arange(batch, device="cuda", dtype=torch.int32) * t_len, n_cached=ints(held),
             n_new=ints(new) if case["ragged"] else None, max_keys=max(total), q=(normal(batch, t_len, hq, d) * case["sharp"] / 2.0).to(torch.bfloat16),
             k_new=(normal(batch, t_len, hkv, d) * loud.reshape(1, 1, hkv, d)).to(torch.bfloat16), v_new=normal(batch, t_len, hkv, d).to(torch.bfloat16),
             out=torch.zeros(batch, t_len, hq, d, dtype=torch.bfloat16, device="cuda"), workspace=torch.zeros(64 << 20, dtype=torch.uint8, device="cuda"))
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import compressed_composable_kv_gb300 as P
        if op == "chunk":
            P.c2kv_attend_pages8_chunk(s["geom"], 0, s["k8"], s["v8"], s["k_scale"], s["v_scale"], s["page_table"], s["n_cached"], s["max_keys"], s["q"],
                                       s["k_new"], s["v_new"], s["rope_table"], s["rope_row"], s["out"], s["workspace"], s["n_new"])
        elif op == "fork":
            P.c2kv_pages8_fork(s["geom"], s["k8"], s["v8"], s["k_scale"], s["v_scale"], s["refs"], s["page_table"], s["n_cached"], s["parent"],
                               s["case"]["room"], s["refs_out"], s["page_table_out"], s["n_cached_out"], s["workspace"])
        else:
            P.c2kv_pages8_compact(s["geom"], s["k8"], s["v8"], s["k_scale"], s["v_scale"], s["refs"], s["page_table"], s["refs_out"], s["page_table_out"],
                                  s["moved_out"], s["workspace"])
    elif op == "chunk":
        n_new = s["n_new"] if s["n_new"] is not None else torch.full_like(s["n_cached"], s["case"]["t_len"])
        _plain_append(s, s["k_new"], s["v_new"], n_new)
        _plain_attend(s, n_new)
    elif op == "fork":
        _plain_fork(s)
    else:
        _plain_compact(s)
    held = {name: s[name] for name in ("k8", "v8", "k_scale", "v_scale")}
    if op == "chunk":
        return dict(held, out=s["out"])
    return dict(held, **{name: s[name] for name in ("refs_out", "page_table_out", "n_cached_out", "moved_out") if name in s})


# ------------------------------------------------------------------ the plain form

def _exponent(a):
    """The smallest e with a <= 448 * 2^e = 1.75 * 2^(8 + e), at least MIN_EXPONENT."""
    m, x = torch.frexp(a)
    return torch.where(2.0 * m <= 1.75, x - 9, x - 8).clamp(min=MIN_EXPONENT).where(a > 0, torch.full_like(x, MIN_EXPONENT))


def _times_power(x, e):
    return (x.double() * torch.exp2(e.double())).float()


def _quantise(x):
    """Codes and scales of [..., page, d] values, one scale for the last two axes."""
    e = _exponent(x.abs().amax((-2, -1)))
    return _times_power(x, -e[..., None, None]).to(torch.float8_e4m3fn), torch.exp2(e.double()).float()


def _rotate(x, cos, sin):
    a, b = x.double().chunk(2, -1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _turns(s):
    """cos and sin, in 64 bits, of each token [batch][t_len][1][d/2]."""
    t = s["rope_table"][s["rope_row"].long()[:, None] + torch.arange(s["case"]["t_len"], device="cuda")].double()[:, :, None]
    return t[..., 0] + t[..., 1], t[..., 2] + t[..., 3]


def _plain_append(s, k_new, v_new, n_new):
    page, table, n = s["case"]["page"], s["page_table"].long(), s["n_cached"].long()
    batch, t_len = k_new.shape[:2]
    k_new = _rotate(k_new, *_turns(s)).float().to(torch.bfloat16)
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
        e = _exponent(x.abs().amax((-2, -1)))
        e_old = torch.frexp(before)[1] - 1
        e = torch.where(has_old, torch.maximum(e, e_old), e)
        coarser = _times_power(was.view(torch.float8_e4m3fn).float(), (e_old - e).clamp(max=0)[..., None, None]).to(torch.float8_e4m3fn)
        new = _times_power(x, -e[..., None, None]).to(torch.float8_e4m3fn)
        raw[at] = torch.where(fresh, new.view(torch.uint8), torch.where(old, coarser.view(torch.uint8), was))
        scales[at] = torch.exp2(e.double()).float()


def _plain_attend(s, n_new):
    table, n = s["page_table"].long().clamp(min=0), s["n_cached"].long()
    batch, t_len, hq, d = s["q"].shape
    q = _rotate(s["q"], *_turns(s)).float()

    def values(codes, scales):
        x = codes[0].view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * scales[0][table][..., None, None]
        return x.transpose(1, 2).reshape(batch, x.shape[2], -1, d)  # [batch][kv head][key][d]

    k = values(s["k8"], s["k_scale"])
    hkv, keys = k.shape[1:3]
    rows = q.reshape(batch, t_len, hkv, -1, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, -1, d)  # [batch][kv head][head of the group, token][d]
    score = (rows @ k.transpose(2, 3) / math.sqrt(d)).reshape(batch, hkv, -1, t_len, keys)
    last = (n[:, None] + torch.arange(t_len, device=n.device))[:, None, None, :, None]
    score.masked_fill_(torch.arange(keys, device=n.device) > last, -math.inf)
    score -= score.amax(-1, keepdim=True)
    p = score.exp_()
    seen = torch.arange(keys, device=n.device) < (n + n_new)[:, None]
    v = torch.where(seen[:, None, :, None], values(s["v8"], s["v_scale"]), 0.0)
    out = (p.reshape(batch, hkv, -1, keys) @ v).reshape(batch, hkv, -1, t_len, d) / p.sum(-1, keepdim=True)
    out = out.permute(0, 3, 1, 2, 4).reshape(batch, t_len, hq, d).to(torch.bfloat16)
    is_new = torch.arange(t_len, device=n.device) < n_new[:, None]
    s["out"].copy_(torch.where(is_new[:, :, None, None], out, s["out"]))


def _plain_fork(s):
    page, room = s["case"]["page"], s["case"]["room"]
    table, n, parent, refs = s["page_table"].long(), s["n_cached"].long(), s["parent"].long(), s["refs"].clone()
    col = torch.arange(table.shape[1], device=table.device)
    is_held = (table >= 0).long().cumprod(1).bool()
    r = parent.clamp(min=0)
    alive = (parent >= 0) & (n[r] >= 0)
    earlier = (r[:, None] == r) & alive & (torch.arange(len(r), device=r.device) < torch.arange(len(r), device=r.device)[:, None])
    first = alive & ~earlier.any(1)
    children = torch.zeros_like(n).index_add_(0, r, alive.long())
    full = n.clamp(min=0) // page
    change = torch.where(col < full[:, None], children[:, None], (children > 0).long()[:, None]) - 1
    refs.index_add_(0, table[is_held], change[is_held].to(refs.dtype))
    keep = torch.where(alive, torch.where(first, is_held.sum(1)[r], full[r]), 0)
    want = torch.where(alive, torch.maximum(keep, (n[r] + room + page - 1) // page), 0)
    new = torch.where(col < keep[:, None], table[r], -1)
    taken = (col >= keep[:, None]) & (col < want[:, None])
    fresh = torch.nonzero(refs == 0)[:, 0][: int(taken.sum())]
    new[taken] = fresh
    refs[fresh] = 1
    copied = alive & ~first & (n[r] % page > 0)
    src, dst = (t[copied].gather(1, full[r][copied][:, None])[:, 0] for t in (table[r], new))
    rows = (torch.arange(page, device=n.device) < (n[r] % page)[copied][:, None])[:, None, :, None]
    for name in "kv":
        raw = s[name + "8"].view(torch.uint8)
        raw[:, dst] = torch.where(rows, raw[:, src], raw[:, dst])
        s[name + "_scale"][:, dst] = s[name + "_scale"][:, src]
    s["refs_out"].copy_(refs)
    s["page_table_out"].copy_(new)
    s["n_cached_out"].copy_(torch.where(alive, n[r], -1))


def _plain_compact(s):
    table, refs = s["page_table"].long(), s["refs"]
    used = refs > 0
    at = torch.arange(len(refs), device=refs.device)
    behind = at >= used.sum()
    src, dst = torch.nonzero(used & behind)[:, 0], torch.nonzero(~used & ~behind)[:, 0]
    moved = torch.where(used, at, -1)
    moved[src] = dst
    for name in "kv":
        raw = s[name + "8"].view(torch.uint8)
        raw[:, dst] = raw[:, src]
        s[name + "_scale"][:, dst] = s[name + "_scale"][:, src]
    s["refs_out"].zero_()
    s["refs_out"][moved[used]] = refs[used]
    is_held = (table >= 0).long().cumprod(1).bool()
    s["page_table_out"].copy_(torch.where(is_held, moved[table.clamp(min=0)], -1))
    s["moved_out"].copy_(moved)


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


def _exact_put(codes, scales, ids, page, first, x):
    """Rows first, first + 1, ... of a sequence get x [head][rows][d]."""
    done = 0
    while done < x.shape[1]:
        row = (first + done) % page
        take = min(page - row, x.shape[1] - done)
        pid = int(ids[(first + done) // page])
        part = x[:, done : done + take]
        scale = _scale_of(part.abs().amax((1, 2)))
        if row:
            scale = torch.maximum(scale, scales[pid])
            codes[pid, :, :row] = _e4m3(codes[pid, :, :row] * (scales[pid] / scale)[:, None, None])
        codes[pid, :, row : row + take] = _e4m3(part / scale[:, None, None])
        scales[pid] = scale
        done += take


def _exact_chunk(s):
    case = s["case"]
    page, hkv, d = case["page"], s["geom"].n_kv_heads, s["geom"].head_dim
    got = {name: s[name].double() for name in ("k8", "v8", "k_scale", "v_scale")}
    out = s["out"].double()
    tables = s["page_table"].tolist()
    for b, (n, t) in enumerate(zip(_lengths(case), _new_lengths(case))):
        if t == 0:
            continue
        rope = s["rope_table"][int(s["rope_row"][b]) :][:t].double()
        turn = torch.complex(rope[..., 0] + rope[..., 1], rope[..., 2] + rope[..., 3])[:, None]

        def turned(x):
            z = torch.complex(x[..., : d // 2], x[..., d // 2 :]) * turn
            return torch.cat((z.real, z.imag), -1)

        k_new = turned(s["k_new"][b, :t].double()).float().to(torch.bfloat16).double()
        _exact_put(got["k8"][0], got["k_scale"][0], tables[b], page, n, k_new.transpose(0, 1))
        _exact_put(got["v8"][0], got["v_scale"][0], tables[b], page, n, s["v_new"][b, :t].double().transpose(0, 1))
        ids = torch.tensor(tables[b][: -(-(n + t) // page)], device="cuda")
        k, v = ((got[x + "8"][0, ids] * got[x + "_scale"][0, ids][..., None, None]).transpose(0, 1).reshape(hkv, -1, d)[:, : n + t] for x in "kv")
        q = turned(s["q"][b, :t].double())
        after = torch.arange(n + t, device="cuda") > n + torch.arange(t, device="cuda")[:, None]
        for h in range(q.shape[1]):
            kv = h // (q.shape[1] // hkv)
            p = torch.softmax((q[:, h] @ k[kv].T * d ** -0.5).masked_fill(after, -math.inf), -1)
            out[b, :t, h] = p @ v[kv]
    return dict(got, out=out)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "chunk":
        return _exact_chunk(s)
    page = case["page"]
    refs, table = s["refs"].tolist(), [[i for i in row if i >= 0] for row in s["page_table"].tolist()]
    width = s["page_table"].shape[1]
    held = {name: s[name].double() for name in ("k8", "v8", "k_scale", "v_scale")}

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def copy(src, dst, rows):
        for x in "kv":
            held[x + "8"][:, dst, :, :rows] = held[x + "8"][:, src, :, :rows]
            held[x + "_scale"][:, dst] = held[x + "_scale"][:, src]

    if case["op"] == "compact":
        used = [i for i, c in enumerate(refs) if c]
        holes = [i for i, c in enumerate(refs[: len(used)]) if not c]
        to = {i: i if i < len(used) else holes.pop(0) for i in used}
        for i in used:
            if to[i] != i:
                copy(i, to[i], page)
        out = [0] * len(refs)
        for i in used:
            out[to[i]] = refs[i]
        return dict(held, refs_out=ints(out), page_table_out=ints([[to[i] for i in row] + [-1] * (width - len(row)) for row in table]),
                    moved_out=ints([to.get(i, -1) for i in range(len(refs))]))
    lens, parents, new = _lengths(case), s["parent"].tolist(), []
    counts = [0] * len(refs)
    for i, r in enumerate(parents):  # what goes on from sequence to sequence
        row = [] if r < 0 else table[r] if r not in parents[:i] else table[r][: lens[r] // page]
        new.append(list(row))
        for x in row:
            counts[x] += 1
    free = [x for x, c in enumerate(counts) if not c]
    for i, r in enumerate(parents):
        if r < 0:
            continue
        tail = lens[r] % page
        if tail and len(new[i]) == lens[r] // page:
            new[i].append(free.pop(0))
            counts[new[i][-1]] = 1
            copy(table[r][lens[r] // page], new[i][-1], tail)
        while len(new[i]) * page < lens[r] + case["room"]:
            new[i].append(free.pop(0))
            counts[new[i][-1]] = 1
    return dict(held, refs_out=ints(counts), page_table_out=ints([row + [-1] * (width - len(row)) for row in new]),
                n_cached_out=ints([lens[r] if r >= 0 else -1 for r in parents]))
