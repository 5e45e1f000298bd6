"""Codes of the cache follow the real quotient x*q/m, ties to even, for every type: each is equal to
the one of the double-precision reference, whose quotients are exact enough to decide (x*q has 33 bits
at most and m 24, so a quotient that is not half way between two codes is more than 2^-40 of itself
from there, where float64 is off by 2^-53).

The rows hold what is hardest: for a group's largest magnitude m, the numbers nearest to each border
between two codes, one step of the type to either side of it, and m itself."""
import numpy as np
import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
from oracle import heads as ref
from test_heads import CODES, DT, f64, make_cache, numbers

pytestmark = pytest.mark.gpu

QMAX = {"e4m3": 448.0, "int8": 127.0, "int4": 7.0}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    nrm.load()


def borders(kind):
    """Half way between neighbouring codes."""
    if kind == "e4m3":
        v = torch.arange(0, 127, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
        return (v[1:] + v[:-1]) / 2
    return np.arange(int(QMAX[kind])) + 0.5


def hard_rows(dtype, kind, tokens, heads, d, group, small):
    """[tokens, heads, d] of which every group holds its largest magnitude and numbers at borders."""
    rng = np.random.default_rng(d + group + len(kind))
    n = tokens * heads * d // group
    low, high = (-14, 15) if dtype == "f16" else (-99, 127)  # m between 2^low and 2^(high + 1)
    m = rng.uniform(1, 2, n) * 2.0 ** rng.integers(low, high + 1, n)
    few = n // 4
    m[:few] = QMAX[kind] * 2.0 ** rng.integers(max(low, -90), min(high, 100) - 9, few)  # ties that the type holds
    if not small:
        m[few:2 * few] = rng.uniform(1, 2, few) * 2.0 ** rng.choice([-37, -36, 99, 100] if dtype != "f16" else [-14, 14], few)
    m = torch.from_numpy(m).clamp(max=torch.finfo(DT[dtype]).max).to(DT[dtype])
    b = torch.from_numpy(rng.choice(borders(kind), (n, group)))
    x = (b * m.double()[:, None] / QMAX[kind]).to(DT[dtype])
    ints = {2: torch.int16, 4: torch.int32}[x.element_size()]
    step = torch.from_numpy(rng.integers(-1, 2, (n, group))).to(ints)
    x = (x.view(ints) + step * (x.view(ints) > 0)).view(DT[dtype])
    x = torch.minimum(x, m[:, None]) * torch.from_numpy(rng.choice([-1.0, 1.0], (n, group))).to(DT[dtype])
    x[torch.arange(n), torch.from_numpy(rng.integers(0, group, n))] = m
    return x.reshape(tokens, heads, d)


@pytest.mark.parametrize("kind", ["e4m3", "int8", "int4"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,group,offset", [(256, 256, 0), (256, 32, 0), (128, 64, 2), (96, 24, 0), (64, 64, 1), (30, 10, 0)])
def test_codes_at_the_borders(dtype, kind, d, group, offset):
    tokens, heads = 200, 2
    rows = [hard_rows(dtype, kind, tokens, heads, d, group, small) for small in (False, True)]
    k, v = (torch.empty(x.numel() + offset, dtype=x.dtype, device="cuda")[offset:].view(x.shape).copy_(x) for x in rows)
    slots = torch.randperm(tokens, generator=torch.Generator().manual_seed(0)).cuda()
    cache = make_cache(kind, tokens // 8, 8, heads, d, group)
    step = make_cache(kind, tokens // 8, 8, heads, d, group)
    nrm.nrm_kv_cache_write(k, v, cache, slots)
    # the serving step without norm or rotation writes the rows themselves
    q = torch.empty_like(k)
    nrm.nrm_qk_norm_rope_cache(k, k, v, None, None, None, None, q, None, step, slots, 1e-6, norm=False)
    nrm.nrm_sync_status()
    for x, n in ((k, "k"), (v, "v")):
        want_c, want_s = ref.quantise(f64(x), kind, group)
        for c in (cache, step):
            got_c = getattr(c, n + "_codes").view(torch.uint8).flatten(0, 1)[slots].view(CODES[kind])
            np.testing.assert_array_equal(numbers(got_c, kind), want_c, err_msg=f"{n} codes")
            np.testing.assert_array_equal(getattr(c, n + "_scales").flatten(0, 1)[slots].cpu().numpy(), want_s)


@pytest.mark.parametrize("kind", ["e4m3", "int8", "int4"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_codes_of_many_rows(dtype, kind):
    # 4 million numbers of ordinary rows
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(8192, 4, 128, device="cuda", generator=g).to(DT[dtype])
    cache = make_cache(kind, 128, 64, 4, 128, 32)
    nrm.nrm_kv_cache_write(x, None, cache, torch.arange(8192, device="cuda"))
    nrm.nrm_sync_status()
    want_c, want_s = ref.quantise(f64(x), kind, 32)
    np.testing.assert_array_equal(numbers(cache.k_codes.flatten(0, 1), kind), want_c)
    np.testing.assert_array_equal(cache.k_scales.flatten(0, 1).cpu().numpy(), want_s)
