"""A wait of the attention over 8-bit pages that runs out, wherever it does: the
launch ends, says so, and leaves its scratch as the next launch needs it."""
import numpy as np
import pytest
import torch

import compressed_composable_kv_gb300 as P
from compressed_composable_kv_gb300 import synth as S
from test_gpu_pages8 import Pool, _dev, _f64, _geom, _ok, _rope, _values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,group", [(128, 1), (128, 4), (64, 2), (64, 8)])
@pytest.mark.parametrize("held", [
    [3000, 700, 90],                        # units shared by many CTAs
    [100] * 6,                              # a unit to a CTA
    [37 * i % 900 + 1 for i in range(90)],  # several units to a CTA
])
def test_a_wait_that_runs_out_in_one_warp_ends_the_launch(d, group, held):
    """The test hook lets every other CTA's wait run out in one of its four
    softmax warps at the last tile of a unit: the warps leave together."""
    g = _geom(d, group, 4)
    pool = Pool(g, 32, [n + 1 for n in held])
    for kv in (0, 1):
        for b, n in enumerate(held):
            pool.put(0, b, 0, kv, _f64(_values(pool.rng, (4, n, d))))
    pool.upload()
    batch = len(held)
    q = _dev(S.normal_bf16(pool.rng, (batch, g.n_q_heads, d)))
    k, v = (_dev(S.normal_bf16(pool.rng, (batch, 4, d))) for _ in range(2))
    n_dev = torch.tensor(held, dtype=torch.int32, device="cuda")
    row = torch.arange(batch, dtype=torch.int32, device="cuda")
    tab, most = _rope(g, np.arange(batch) * 17), max(held) + 1
    ws = torch.zeros(P.c2kv_attend_pages8_workspace_size(g, batch, most), dtype=torch.uint8, device="cuda")
    out = torch.empty((batch, g.n_q_heads, d), dtype=torch.bfloat16, device="cuda")

    def step():
        P.c2kv_attend_pages8(g, 0, *pool.args(), n_dev, most, q, k, v, tab, row, out, ws)
        torch.cuda.synchronize()
        return out.clone()

    good = step()
    _ok()
    for _ in range(2):
        P.c2kv_test_expire_next_waits(1)
        step()
        P.c2kv_test_expire_next_waits(0)
        assert P.c2kv_device_error() == P.C2KV_ETIMEOUT
        assert (ws[: 256 * 4 * 4].view(torch.int32) == 0).all(), "counters are not back at zero"
        assert torch.equal(step(), good)
        _ok()
