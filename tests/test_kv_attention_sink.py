"""Attention over the paged cache where a position draws nearly all of the weight and has next to no
value, so that the output is made of weights far below the largest.  Against the double-precision
reference, with the tolerances of test_kv_attention_long.py.
"""
import numpy as np
import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
from test_heads import DT, f64
from test_kv_attention import Case
from test_kv_attention_long import _gpu, check_rows  # noqa: F401

pytestmark = pytest.mark.gpu


def held(t, at, head):
    return t.cpu()[at[0], at[1], head]


def check_sequence(c, s, out, lse, scale, tiles, exact=()):
    j = np.arange(int(c.lengths[s]))
    at = (c.table[s, j // c.page], j % c.page)
    heads = c.hq // c.hk
    for g in range(c.hk):
        rows = slice(g * heads, (g + 1) * heads)
        codes = [held(t.view(torch.uint8), at, g).contiguous().view(t.dtype) for t in c.codes]
        if c.kind == "e4m3":
            codes = [t.float() for t in codes]
        check_rows(c.dtype, c.kind, f64(c.q)[s, rows], *((codes[t].numpy(), held(c.scales[t], at, g).numpy()) for t in range(2)),
                   scale, f64(out)[s, rows], f64(lse)[s, rows], tiles, exact)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind,d,group", [("e4m3", 64, 64), ("e4m3", 128, 32), ("int8", 64, 16), ("int4", 128, 32), ("e4m3", 256, 256),
                                          ("int8", 128, 128), ("e4m3", 40, 8), ("int4", 40, 8)])
@pytest.mark.parametrize("above", [12, 16, 20, 25])
@pytest.mark.parametrize("value", ["none", "codes of zero", "small"])
def test_a_position_that_draws_the_weight_and_has_no_value(dtype, kind, d, group, above, value):
    for others in (30, 600):
        c = Case(dtype, [others + 1], 12, 2, d, kind, group, 16, poison=0.0)
        page, slot = int(c.table[0, 0]), 0
        scale = d ** -0.5
        sign = torch.where(torch.randn(d, generator=torch.Generator().manual_seed(others)) > 0, 1.0, -1.0)
        c.q = (sign * (1 - torch.arange(12)[:, None] / 32)).to(DT[dtype])[None]
        # its key is 4 times the queries' signs, the others' keys are small: a logit of `above`, and of about 0.1
        code = 4 * sign
        if kind == "int4":
            low, high = (code[i::2].long() & 15 for i in range(2))
            code = (low | high << 4)
        c.scales[0].mul_(0.1)
        c.codes[0][page, slot] = code.to(c.codes[0].dtype).cuda()
        c.scales[0][page, slot] = above / (scale * 4 * d)
        # values of one sign: they do not cancel; in float16 large enough not to fall among its smallest numbers
        c.scales[1].mul_(2.0 ** 12 if dtype == "f16" else 1)
        if kind == "e4m3":
            c.codes[1].view(torch.uint8).bitwise_and_(0x7f)
        else:
            c.codes[1].bitwise_and_(0x77 if kind == "int4" else 0x7f)
        if value == "none":
            c.scales[1][page, slot] = 0
        elif value == "small":
            c.scales[1][page, slot] *= 2.0 ** -14
        else:
            c.codes[1].view(torch.uint8)[page, slot] = 0
        out, lse = c.run(lse=True, scale=scale)
        nrm.nrm_sync_status()
        check_sequence(c, 0, out, lse, scale, others // 32 + 1, exact=[0])
