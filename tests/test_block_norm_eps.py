"""The norms around a block with an eps so small that the third power of a row's statistic leaves
float32: the reference and the tolerances of test_block_norm.py."""
import pytest
import torch

import test_block_norm as tb
from test_block_norm import _gpu  # noqa: F401

pytestmark = pytest.mark.gpu


# rows of whole vectors, of any length, and too long for either; a gate for all rows, for some, for each
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols,gates", [(512, 0), (4096, 1), (520, 6), (256, 36), (333, 1), (67, 36), (12000, 2), (9001, 1)])
def test_small_eps(dtype, cols, gates, monkeypatch):
    monkeypatch.setattr(tb, "EPS", 1e-30)
    b = tb.Block(dtype, 36, cols, gates)
    b.f[3] = 0
    b.x[3] = 0
    for t in (b.x, b.f):
        t[:30] *= 1e-14
        t[5] *= 1e-3
    # (the stream after the block is x and f's norm: of the same size)
    b.w_post *= 1e-14
    b.check()
