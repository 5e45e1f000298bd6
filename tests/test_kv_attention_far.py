"""Attention over sequences of more than 2^32 positions, whose pages are the few of a small cache many
times over: positions do not fit the 32 bits that the cache's slots do."""
import re

import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
from test_dependent_launch import code
from test_heads import same


def test_positions_are_divided_as_far_as_they_reach():
    # the division by multiplication holds for what is below its bound, and positions reach the table's width
    text = code("kvattn_api.cu")
    call = text[text.index("nrm_status nrm_kv_cache_attention("):]
    assert re.search(r"a\.cache\.page = make_row_div\(cache->page_size, std::max\(a\.cache\.slots, a\.cap\)\);", call)


@pytest.mark.gpu
@pytest.mark.parametrize("d,group", [(16, 16), (10, 10)])
@pytest.mark.parametrize("past", [50, -7, 1 << 19])
def test_positions_beyond_32_bits(d, group, past):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    page, g = 1 << 20, torch.Generator(device="cuda").manual_seed(d)
    codes = [torch.randint(-127, 128, (5, page, 1, d), generator=g, device="cuda").to(torch.int8) for _ in range(2)]
    scales = [torch.rand(5, page, 1, d // group, generator=g, device="cuda") / 60 for _ in range(2)]
    cache = nrm.kv_cache(codes[0], scales[0], codes[1], scales[1])
    q = torch.randn(2, 4, d, generator=g, device="cuda")
    far = torch.randint(0, 5, (2, (1 << 12) + 1), generator=g, device="cuda")
    outs = []
    for skipped in (0, 1 << 12):  # whole, and its last pages alone
        table = far[:, skipped - 1:].contiguous() if skipped else far
        before = (skipped - 1) * page if skipped else 0
        lengths = torch.tensor([(1 << 32) + past - before, (1 << 32) + past // 2 - before], device="cuda")
        out, lse = torch.empty_like(q), torch.empty(2, 4, device="cuda")
        nrm.nrm_kv_cache_attention(q, cache, table, lengths, out, d ** -0.5, nrm.kv_attention_workspace(q, cache, table),
                                   window=1000, lse=lse)
        nrm.nrm_sync_status()
        outs.append((out, lse))
    assert same(outs[0][0], outs[1][0]) and same(outs[0][1], outs[1][1])
    assert outs[0][0].isfinite().all() and outs[0][0].any()
