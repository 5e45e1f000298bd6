"""Seeded random shapes of the operators on heads, beside the fixed ones of test_heads.py: types, heads,
rows from 1 to 256 elements, rotations and pair layouts, axes, strides and offsets, cache groups, pages
and layouts.  What decides between the paths depends on all of these at once.  Each case draws its
parameters from its own seed; the comparisons and their tolerances are those of test_heads.py, and the
serving step's are stated here."""
import math

import numpy as np
import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
import test_heads as H
from oracle import heads as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    nrm.load()


def _log_uniform(r, lo, hi):
    return int(min(hi, max(lo, round(math.exp(r.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(seed, even=False):
    """dtype, tokens, hq, hk, d, rot, pairs, axes, fused, offset"""
    r = np.random.default_rng(seed)
    dtype = str(r.choice(["f32", "f16", "bf16"]))
    d = int(r.choice([r.integers(1, 257), 2 * r.integers(1, 129), 4 * r.integers(1, 65), 8 * r.integers(1, 33),
                      16 * r.integers(1, 17), 2 ** r.integers(3, 9)]))
    if even and d % 2:
        d += 1
    rot = int(r.choice([d // 2 * 2, 2 * r.integers(0, d // 2 + 1), d // 4 * 2, d // 16 * 8]))
    hk = _log_uniform(r, 1, 8)
    hq = int(r.choice([hk, hk * r.integers(1, 5), r.integers(1, 20)]))
    tokens = _log_uniform(r, 1, max(1, min(5000, (1 << 20) // ((hq + hk) * d), 40000 // max(1, rot // 2))))
    return (dtype, tokens, hq, hk, d, rot, str(r.choice(["half", "pair"])), int(r.integers(1, 5)) if rot else 1,
            bool(r.random() < 0.5), int(r.choice([0, 0, 0, 0, 1, 2, 4]))), r


def draw_cache(seed):
    kind = ("e4m3", "int8", "int4")[seed % 3]
    shape, r = draw(seed, even=kind == "int4")
    d = shape[4]
    groups = [n for n in range(1, d + 1) if d % n == 0 and (kind != "int4" or n % 2 == 0)]
    return shape, kind, int(r.choice([d, r.choice(groups), r.choice(groups[-3:])])), int(r.integers(1, 70)), str(
        r.choice(["token", "head", "joined"])), r


@pytest.mark.parametrize("case", range(48))
def test_fuzz_norm_and_rotation(case):
    shape, r = draw(9300 + case)
    H.test_norm_rope_forward_and_backward(*shape, bool(r.random() < 0.7))


@pytest.mark.parametrize("case", range(32))
def test_fuzz_rotation(case):
    H.test_rope_forward_backward_and_in_place(*draw(9400 + case)[0])


def check_cache(cache, kind, group, slots, rows, back):
    """Codes and scales of `rows` (k, v) at `slots` are the reference's, and read back as their values."""
    live = slots >= 0
    if not live.any():
        assert not any(b.any() for b in back)
        return
    for x, n, got in zip(rows, "kv", back):
        want_c, want_s = ref.quantise(H.f64(x[live]), kind, group)
        codes, scales = getattr(cache, n + "_codes"), getattr(cache, n + "_scales")
        np.testing.assert_array_equal(H.numbers(H.at_slots(codes, slots[live]), kind), want_c, err_msg=n)
        np.testing.assert_array_equal(H.at_slots(scales, slots[live]).cpu().numpy(), want_s, err_msg=n)
        value = torch.from_numpy(want_c).float().unflatten(-1, (-1, group)) * torch.from_numpy(want_s)[..., None]
        value = value.flatten(-2).to(got.dtype)
        assert torch.equal(got[live].cpu().isnan(), value.isnan()) and not got[~live].any()
        assert torch.equal(got[live].cpu().nan_to_num(), value.nan_to_num())


@pytest.mark.parametrize("case", range(48))
def test_fuzz_cache(case):
    # codes, scales and values bit for bit; rows of zeros, of ties, with a NaN and an infinity; the
    # slots that no token names stay as they were
    (dtype, tokens, _, hk, d, _, _, _, fused, offset), kind, group, page, layout, r = draw_cache(9500 + case)
    c = H.Data(dtype, tokens, hk, hk, d, 0, fused=fused, offset=offset)
    if tokens > 8:
        c.k[0] = 0
        c.k[1] = torch.arange(d, device="cuda").remainder(16).to(c.k.dtype) - 8
        c.k[2, 0, d // 2] = float("nan")
        c.k[3, 0, 0] = float("-inf")
        c.k[4] *= 1e-3
    pages = -(-tokens // page) + 2
    cache = H.make_cache(kind, pages, page, hk, d, group, layout)
    before = {n: getattr(cache, n).clone() for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(case))[:tokens].cuda()
    slots[torch.from_numpy(r.random(tokens) < 0.1).cuda()] = -1
    nrm.nrm_kv_cache_write(c.k, c.v, cache, slots)
    back = [H.Guarded((tokens, hk, d), H.DT[dtype], offset * c.k.element_size()) for _ in range(2)]
    for b in back:
        b.t.zero_()
    nrm.nrm_kv_cache_read(cache, slots, back[0].t, back[1].t)
    nrm.nrm_sync_status()
    for b in back:
        b.check("read")
    check_cache(cache, kind, group, slots, (c.k, c.v), [b.t for b in back])
    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    rest[slots[slots >= 0]] = False
    rest = rest.nonzero().flatten()
    for n, t in before.items():
        assert H.same(H.at_slots(getattr(cache, n).view(torch.uint8), rest), H.at_slots(t.view(torch.uint8), rest)), n


@pytest.mark.parametrize("case", range(48))
def test_fuzz_serving_step(case):
    # q_out and k_out within the bounds of the separate calls (24 u of a normed pair, 8 u of a turned one);
    # the cache holds the codes of the key that the call itself returns, and of the value, bit for bit;
    # the same without the key, and read back
    (dtype, tokens, hq, hk, d, rot, pairs, axes, fused, offset), kind, group, page, layout, r = draw_cache(9600 + case)
    norm = bool(r.random() < 0.6)
    c = H.Data(dtype, tokens, hq, hk, d, rot, axes, fused, offset, seed=2)
    pages = -(-tokens // page) + 1
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(case))[:tokens].cuda()
    slots[torch.from_numpy(r.random(tokens) < 0.1).cuda()] = -1
    caches = [H.make_cache(kind, pages, page, hk, d, group, layout) for _ in range(2)]
    outs = [[H.Guarded((tokens, h, d), H.DT[dtype], offset * c.q.element_size()) for h in (hq, hk)] for _ in range(2)]
    for i, (cache, (qo, ko)) in enumerate(zip(caches, outs)):
        nrm.nrm_qk_norm_rope_cache(c.q, c.k, c.v, c.wq, c.wk, c.pos, c.inv, qo.t, None if i else ko.t, cache, slots, 1e-5,
                                   axis=c.axis, pairs=pairs, norm=norm)
        nrm.nrm_sync_status()
        qo.check("q_out"), ko.check("k_out")
    ang = c.angles()
    for x, w, got, tag in ((c.q, c.wq, outs[0][0].t, "q_out"), (c.k, c.wk, outs[0][1].t, "k_out")):
        x = H.f64(x)
        if norm:
            want, rr = ref.norm_rope_fwd(x, H.f64(w), ang, 1e-5, pairs)
            size, n = x * rr[..., None] * H.f64(w), 24
        else:
            want, size, n = ref.rotate(x, ang, pairs), x, 8
        H.within(got, want, n * H.U * ref.pair_size(size, rot // 2, pairs), dtype, tag)
    assert H.same(outs[0][0].t, outs[1][0].t)
    back = [torch.zeros(tokens, hk, d, dtype=H.DT[dtype], device="cuda") for _ in range(2)]
    nrm.nrm_kv_cache_read(caches[1], slots, *back)
    nrm.nrm_sync_status()
    for cache in caches:
        check_cache(cache, kind, group, slots, (outs[0][1].t, c.v), back)
