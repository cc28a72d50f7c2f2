"""Chunk attention over the 8-bit pages at the ends of its range, against the fp64
oracle (oracle/pages8_oracle.py): units of one tile, many to a CTA."""
import pytest

from test_gpu_chunk8 import Chunk
from test_gpu_pages8 import _geom, _ok

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
