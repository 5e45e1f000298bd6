"""Attention over the paged cache with scales and queries at the ends of float32: the reference and the
tolerances of test_kv_attention.py."""
import pytest
import torch

from test_heads import DT
from test_kv_attention import Case, _gpu  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [("f32", 64, 16), ("bf16", 64, 64), ("f32", 128, 32), ("bf16", 256, 64), ("f32", 40, 8), ("bf16", 40, 40)]


@pytest.mark.parametrize("kind", ["e4m3", "int8", "int4"])
@pytest.mark.parametrize("dtype,d,group", SHAPES)
@pytest.mark.parametrize("size", [60, 100, 116])
def test_large_scales_of_keys(dtype, d, group, kind, size):
    # keys up to 2^118 with queries, or with queries and a scale, so small that the logits are ordinary
    c = Case(dtype, [100, 33, 700], 8, 2, d, kind, group, 16, loud=2.0 ** -size, poison=0.0)
    c.scales[0].mul_(2.0 ** 116)
    scale = d ** -0.5 * 2.0 ** (size - 116)
    c.check(weights=True, scale=scale)
    # among ordinary ones, whose logits are then 0
    c.scales[0][:, ::3] *= 2.0 ** -116
    c.check(weights=True, scale=scale)


@pytest.mark.parametrize("kind", ["e4m3", "int8", "int4"])
@pytest.mark.parametrize("dtype,d,group", SHAPES)
@pytest.mark.parametrize("size", [124, -125])
def test_queries_at_the_ends_of_float32(dtype, d, group, kind, size):
    # (float32 and bfloat16 reach from 2^-126 to 2^128)
    c = Case(dtype, [100, 33, 300], 8, 2, d, kind, group, 16, loud=2.0 ** size, poison=0.0)
    c.scales[0].mul_(2.0 ** (-60 if size > 0 else 60))
    c.check(weights=True, scale=d ** -0.5 * 2.0 ** (-size + (60 if size > 0 else -60)))


@pytest.mark.parametrize("dtype,d,group", SHAPES)
@pytest.mark.parametrize("kind", ["e4m3", "int8", "int4"])
def test_the_largest_queries_and_values(dtype, d, group, kind):
    c = Case(dtype, [70], 4, 2, d, kind, group, 16, poison=0.0)
    most = torch.finfo(DT[dtype]).max
    c.q = torch.where(torch.rand(c.q.shape, generator=torch.Generator().manual_seed(0)) < 0.5, most, -most).to(DT[dtype])
    c.scales[0].mul_(2.0 ** -64)
    c.scales[1].mul_(2.0 ** (120 if kind == "e4m3" else 122) / 16)
    c.check(scale=d ** -0.5 * 2.0 ** -64)
