"""The top alternatives of logits where NaN, large logits and bounds meet
(c2kv_token_logprobs), against the fp64 oracle: indices are equal, and a row
that holds NaN answers NaN."""
import numpy as np
import pytest
import torch

import oracle.pages8_oracle as Q
import compressed_composable_kv_gb300 as P

pytestmark = pytest.mark.gpu


def _run(x, k):
    rows = x.shape[0]
    ent = torch.empty(rows, device="cuda")
    ids, tops = torch.empty((rows, k), dtype=torch.int32, device="cuda"), torch.empty((rows, k), device="cuda")
    P.c2kv_token_logprobs(x, None, k, None, ent, ids, tops)
    return ent, ids, tops


def _nan_rows(vocab, k, seed):
    """Rows with few NaN: one in the middle, one late, one in each part of the
    row; k of them scattered, a few more than k, many more; k in neighbouring
    places; a few in rows that rise along the row, +inf among them."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(14, vocab, generator=gen) * 3
    some = lambda n, lo=0: lo + torch.randperm(vocab - lo, generator=gen)[:n]   # noqa: E731
    x[0, vocab // 2] = torch.nan
    x[1, vocab - 2] = torch.nan
    x[2, vocab // 9] = torch.nan
    x[3, torch.arange(1, 16) * (vocab // 16) + 5] = torch.nan
    x[4, some(k)] = torch.nan
    x[5, some(k + 3)] = torch.nan
    x[6, some(k, vocab // 2)] = torch.nan
    x[7, some(min(8 * k + 100, vocab // 2))] = torch.nan
    x[8, vocab // 3: vocab // 3 + k] = torch.nan
    x[9] = torch.arange(vocab) / 1000.0
    x[9, some(k + 2)] = torch.nan
    x[10] = torch.arange(vocab) / 1000.0
    x[10, some(200, vocab // 3)] = torch.nan
    x[11, some(40)] = torch.inf
    x[11, some(2)] = torch.nan
    x[12] = -torch.inf
    x[12, some(k)] = torch.nan
    x[13] = torch.finfo(torch.bfloat16).min
    x[13, some(1)] = torch.nan
    return x


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [9001, 50257, 128256])
@pytest.mark.parametrize("k", [1, 2, 5, 20, 64])
@pytest.mark.parametrize("copies", [1, 25])   # several CTAs to a row; one
def test_a_few_nan_rank_first(dtype, vocab, k, copies):
    x = _nan_rows(vocab, k, vocab + k).to(dtype)
    _, _, want, _ = Q.token_logprobs(x.double().numpy(), None, k)
    ent, ids, tops = _run(x.cuda().repeat(copies, 1), k)
    got = ids.cpu().numpy().reshape(copies, *want.shape)
    bad = sorted({int(r) for r in np.argwhere((got != want).any((0, 2)))[:, 0]})
    assert not bad, f"rows {bad}: {got[0, bad[0]][:6]} for {want[bad[0]][:6]}"
    assert ent.isnan().all() and tops.isnan().all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [2, 320])   # several CTAs to a row; one
def test_rows_whose_notes_run_over_behind_their_first_step(dtype, rows):
    """A first step whose notes fit, a second one (and every later one) whose
    notes do not: every launch decides alike, and right."""
    vocab, k = 300000, 7
    step = 2048 * 128 // torch.finfo(dtype).bits   # logits of a CTA's step
    gen = torch.Generator().manual_seed(rows)
    x = torch.randn(2, vocab, generator=gen)
    x[0] += 3 * (torch.arange(vocab) // step)
    x[1, step:] += 6.0
    x = x.to(dtype)
    _, _, want, _ = Q.token_logprobs(x.double().numpy(), None, k)
    big = x.cuda().repeat(rows // 2, 1)
    runs = [_run(big, k)[1] for _ in range(20)]
    want = torch.from_numpy(want).cuda().repeat(rows // 2, 1)
    assert all(torch.equal(r, want) for r in runs)
