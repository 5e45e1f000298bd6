"""The backward of the norms around a block passes rows through slots of shared memory that copies
overwrite once their readers have said that they are done: that they say so only after all their
reads is checked in the source without a GPU; on one, rows of one warp each, which say so most
often, go through every slot hundreds of times."""
import re

import pytest
import torch

from test_block_norm import Block, same
from test_dependent_launch import code, kernels


def test_a_slot_is_freed_only_behind_a_barrier():
    body, = [b for s, b in kernels(code("blocknorm.cuh")) if "block_bwd_ring_kernel" in s]
    reads = body.index("dyr[k][j] = in_slot(")
    free = body.index("mbar_arrive(&empty[slot])", reads)
    between = body[reads:free]
    # groups of several warps meet at a named barrier, with and without the sums; one warp, whose sums are
    # exchanges alone, at a barrier that depends on nothing else
    assert "group_sums<ROWS>" in between and "named_barrier(kBlockBar + group, threads)" in between
    assert re.search(r"if \(warps == 1\) __syncwarp\(\);\s*if \(t == 0\) $", between)
    # the other place is a group's without a row in the slot: it has read nothing
    rest = body[free + 1:]
    assert rest.count("mbar_arrive(&empty[slot])") == 1 and "in_slot(" not in rest


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,cols", [("bf16", 256), ("bf16", 64), ("bf16", 67), ("f16", 192), ("f32", 128), ("f32", 63)])
@pytest.mark.parametrize("gates", [0, 1, 4])
def test_rows_of_one_warp_many_times_over(dtype, cols, gates):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    b = Block(dtype, 40000, cols, gates)
    y, _, r1, r2 = b.fwd()
    first = b.bwd(y, r1, r2)
    for _ in range(5):
        assert all(p is None or same(p, q) for p, q in zip(first, b.bwd(y, r1, r2)))
    Block(dtype, 4000, cols, gates).check()
