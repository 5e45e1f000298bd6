"""The operators on attention heads without a GPU: the reference against central
differences and closed forms, the axis map, and every refusal of the C entry
points and of the binding (all before anything is enqueued)."""
import ctypes

import numpy as np
import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
from normalization_layernorm_rmsnorm_gb300 import _binding as B
from normalization_layernorm_rmsnorm_gb300 import build as nbuild
from oracle import heads as ref


@pytest.fixture(scope="module")
def lib():
    nbuild.build()
    return nrm.load()


# ---------------------------------------------------------------------------
# the reference
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("pairs", ["half", "pair"])
@pytest.mark.parametrize("d,rot", [(8, 8), (7, 4), (6, 0)])
def test_reference_gradients_against_differences(pairs, d, rot):
    rng = np.random.default_rng(d + rot)
    x, dy = rng.normal(size=(3, 2, d)), rng.normal(size=(3, 2, d))
    w = 1 + 0.1 * rng.normal(size=d)
    ang = ref.angles(np.array([0, 5, 1000]), 0.5 ** np.arange(rot // 2))
    dx, dw = ref.norm_rope_bwd(dy, x, w, ang, 1e-3, pairs)
    h = 1e-6

    def loss(xx, ww):
        return (ref.norm_rope_fwd(xx, ww, ang, 1e-3, pairs)[0] * dy).sum()

    # central differences: truncation h^2 and rounding 1e-16 / h, both far below 1e-7
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    for i in range(d):
        e = np.zeros_like(w)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_reference_rotation_closed_forms():
    x = np.array([[[3.0, 4.0, 5.0]]])
    quarter = np.array([[np.pi / 2]])
    np.testing.assert_allclose(ref.rotate(x, quarter), [[[-4.0, 3.0, 5.0]]], atol=1e-15)
    np.testing.assert_allclose(ref.rotate(x, quarter, inverse=True), [[[4.0, -3.0, 5.0]]], atol=1e-15)
    # a rotation keeps lengths, and turning back gives the input
    rng = np.random.default_rng(0)
    x, ang = rng.normal(size=(4, 3, 10)), rng.normal(size=(4, 5))
    for pairs in ("half", "pair"):
        y = ref.rotate(x, ang, pairs)
        np.testing.assert_allclose((y * y).sum(-1), (x * x).sum(-1), rtol=1e-13)
        np.testing.assert_allclose(ref.rotate(y, ang, pairs, inverse=True), x, atol=1e-14)


def test_reference_angles_of_far_positions():
    # frequency 1: position n turns by n radians; 2^40 positions on, reduced exactly
    got = ref.angles(np.array([1, 7, 2 ** 40]), np.array([1.0]))[:, 0]
    assert abs(got[0] - 1) < 1e-15 and abs(got[1] - (7 - 2 * np.pi)) < 1e-14
    import math
    assert abs(math.cos(got[2]) - math.cos(2.0 ** 40)) < 1e-9  # libm reduces its argument exactly too


@pytest.mark.parametrize("kind,top", [("e4m3", 448), ("int8", 127), ("int4", 7)])
def test_reference_quantisation_closed_forms(kind, top):
    # the largest magnitude takes the last code; half of it is a tie for the integers, to even
    codes, scale = ref.quantise(np.array([2.0, -1.0, 0.0, 1.0]), kind, 4)
    half = {"e4m3": 224, "int8": 64, "int4": 4}[kind]
    np.testing.assert_array_equal(codes, [top, -half, 0, half])
    assert scale[0] == np.float32(2.0 / top)
    codes, scale = ref.quantise(np.array([0.0, 0.0, 2.0 ** -101, 0.0, np.nan, 1.0, np.inf, 3.0]), kind, 2)
    np.testing.assert_array_equal(codes, np.zeros(8))
    assert scale[0] == 0 and scale[1] == 0 and np.isnan(scale[2]) and np.isnan(scale[3])


def test_e4m3_reference_matches_torch_on_every_value():
    u = torch.linspace(-448, 448, 200_001, dtype=torch.float32)
    u = torch.cat([u, u / 1000, u / 100_000])
    want = u.to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref._round_e4m3(u.double().numpy()), want)


def test_rope_axis():
    assert nrm.rope_axis([2, 3]) == b"\0\0\1\1\1"
    assert nrm.rope_axis([3, 1, 2], interleaved=True) == b"\0\1\2\0\2\0"
    assert nrm.rope_axis([4]) == b"\0\0\0\0"


# ---------------------------------------------------------------------------
# refusals of the C entry points
# ---------------------------------------------------------------------------

P = 1 << 20  # an aligned, non-null address that is never read: every call below is refused on the host


def H(data=P, heads=2, ts=32, hs=16):
    return B._Heads(data, heads, ts, hs)


def R(pos=P, stride=8, inv=P, axis=None, rot=16, axes=1, pairs=0):
    return B._Rope(pos, stride, inv, axis, rot, axes, pairs)


def C(**k):
    a = dict(k_codes=P, k_scales=P, v_codes=2 * P, v_scales=2 * P, pages=4, page_size=8, heads=2, d=16, group=16,
             page_stride=256, slot_stride=32, head_stride=16, scale_page_stride=16, scale_slot_stride=2,
             scale_head_stride=1, kind=1)
    a.update(k)
    return B._Cache(*(a[n] for n, _ in B._Cache._fields_))


def fwd(lib, q=None, k=None, r=None, qo=None, ko=None, wq=None, rq=None, tokens=8, d=16, eps=1e-6, dt=0):
    return lib.nrm_qk_norm_rope_fwd(q or H(), k, wq, None, r, qo or H(3 * P), ko, rq, None, tokens, d, eps, dt, None)


def bwd(lib, dqo=None, q=None, dq=None, k=None, dko=None, dk=None, rq=P, rk=None, dwq=None, dwk=None, ws=None, nws=0,
        r=None, d=16):
    return lib.nrm_qk_norm_rope_bwd(dqo or H(2 * P), dko, q or H(), k, None, None, rq, rk, r, dq or H(3 * P), dk, dwq,
                                    dwk, 8, d, 0, ws, nws, None)


def write(lib, k=H(), v=None, c=None, slots=P, tokens=8, dt=0):
    return lib.nrm_kv_cache_write(k, v, c or C(), slots, tokens, dt, None)


def read(lib, k=H(), v=None, c=None, slots=P, tokens=8, dt=0):
    return lib.nrm_kv_cache_read(c or C(), slots, k, v, tokens, dt, None)


def fused(lib, q=None, k=None, v=None, qo=None, ko=None, c=None, slots=P, r=None, eps=1e-6, d=16, norm=1):
    return lib.nrm_qk_norm_rope_cache(q or H(), k if k is not None else H(2 * P), v or H(4 * P), None, None, r,
                                      qo or H(3 * P), ko, c or C(), slots, 8, d, eps, norm, 0, None)


@pytest.mark.parametrize("call,expect", [
    # sizes and types
    (lambda L: fwd(L, d=0), 1),
    (lambda L: fwd(L, d=257), 2),
    (lambda L: fwd(L, tokens=-1), 1),
    (lambda L: fwd(L, tokens=1 << 40), 2),
    (lambda L: fwd(L, dt=3), 1),
    (lambda L: fwd(L, eps=0.0), 1),
    (lambda L: fwd(L, eps=float("nan")), 1),
    # views: missing, no heads, misaligned, negative or far strides, overlapping rows
    (lambda L: L.nrm_qk_norm_rope_fwd(None, None, None, None, None, H(), None, None, None, 8, 16, 1e-6, 0, None), 1),
    (lambda L: fwd(L, q=H(data=None)), 1),
    (lambda L: fwd(L, q=H(heads=0)), 1),
    (lambda L: fwd(L, q=H(data=P + 2)), 1),
    (lambda L: fwd(L, q=H(ts=-32)), 1),
    (lambda L: fwd(L, q=H(ts=1 << 41)), 1),
    (lambda L: fwd(L, tokens=1 << 30, q=H(ts=1 << 39)), 1),
    (lambda L: fwd(L, qo=H(3 * P, ts=31)), 1),
    (lambda L: fwd(L, qo=H(3 * P, hs=15)), 1),
    (lambda L: fwd(L, qo=H(3 * P, heads=3, ts=48)), 1),
    (lambda L: fwd(L, k=H(2 * P)), 1),  # k without k_out
    # an output on another tensor, or on its own input with other strides
    (lambda L: fwd(L, qo=H(ts=64)), 1),
    (lambda L: fwd(L, k=H(3 * P), ko=H(4 * P)), 1),
    (lambda L: fwd(L, k=H(2 * P), ko=H()), 1),
    (lambda L: fwd(L, k=H(2 * P), ko=H(3 * P)), 1),
    (lambda L: fwd(L, wq=P + 1), 1),
    (lambda L: fwd(L, rq=P + 2), 1),
    (lambda L: L.nrm_qk_norm_rope_fwd(H(), H(2 * P), None, None, None, H(3 * P), H(4 * P), P, P, 8, 16, 1e-6, 0, None), 1),
    # rotations
    (lambda L: fwd(L, r=R(rot=15)), 1),
    (lambda L: fwd(L, r=R(rot=18)), 1),
    (lambda L: fwd(L, r=R(rot=-2)), 1),
    (lambda L: fwd(L, r=R(axes=0)), 1),
    (lambda L: fwd(L, r=R(axes=5, axis=bytes(8))), 1),
    (lambda L: fwd(L, r=R(axes=2)), 1),
    (lambda L: fwd(L, r=R(axes=2, axis=bytes([0, 1, 2, 0, 0, 0, 0, 0]))), 1),
    (lambda L: fwd(L, r=R(axes=2, axis=bytes(8), stride=7)), 1),
    (lambda L: fwd(L, r=R(pairs=2)), 1),
    (lambda L: fwd(L, r=R(pos=None)), 1),
    (lambda L: fwd(L, r=R(inv=None)), 1),
    (lambda L: fwd(L, r=R(pos=P + 4)), 1),
    (lambda L: L.nrm_rope_fwd(H(), None, R(rot=3), H(3 * P), None, 8, 16, 0, None), 1),
    (lambda L: L.nrm_rope_bwd(H(), H(2 * P), R(), H(3 * P), None, 8, 16, 0, None), 1),
    # backward: statistics, in place, a weight gradient without its input
    (lambda L: bwd(L, rq=None), 1),
    (lambda L: bwd(L, dq=H()), 1),
    (lambda L: bwd(L, dq=H(2 * P)), 1),
    (lambda L: bwd(L, dwk=P), 1),
    (lambda L: bwd(L, k=H(4 * P), dko=H(5 * P), dk=H(6 * P), rk=P, dwq=P, dwk=P), 1),
    (lambda L: bwd(L, k=H(4 * P), dko=H(5 * P), dk=H(6 * P)), 1),
    (lambda L: bwd(L, k=H(4 * P), dko=H(5 * P), dk=H(3 * P), rk=P), 1),
    (lambda L: bwd(L, r=R(rot=17)), 1),
    # cache
    (lambda L: write(L, c=C(kind=3)), 1),
    (lambda L: write(L, c=C(pages=0)), 1),
    (lambda L: write(L, c=C(group=5)), 1),
    (lambda L: write(L, c=C(group=0)), 1),
    (lambda L: write(L, c=C(d=15, group=15, kind=2)), 1),
    (lambda L: write(L, c=C(d=300, group=300)), 2),
    (lambda L: write(L, c=C(head_stride=15)), 1),
    (lambda L: write(L, c=C(slot_stride=31)), 1),
    (lambda L: write(L, c=C(page_stride=255)), 1),
    (lambda L: write(L, c=C(scale_slot_stride=1)), 1),
    (lambda L: write(L, c=C(page_stride=-256)), 1),
    (lambda L: write(L, c=C(k_codes=None)), 1),
    (lambda L: write(L, c=C(k_scales=P + 2)), 1),
    (lambda L: write(L, k=None), 1),
    (lambda L: write(L, v=H(2 * P), c=C(v_codes=P)), 1),
    (lambda L: write(L, v=H(2 * P), c=C(v_scales=P)), 1),
    (lambda L: fused(L, c=C(v_codes=P)), 1),
    (lambda L: write(L, k=H(heads=3)), 1),
    (lambda L: write(L, slots=None), 1),
    (lambda L: write(L, slots=P + 4), 1),
    (lambda L: L.nrm_kv_cache_write(H(), None, None, P, 8, 0, None), 1),
    (lambda L: write(L, tokens=-1), 1),
    (lambda L: write(L, dt=4), 1),
    (lambda L: read(L, k=H(ts=8)), 1),
    (lambda L: read(L, v=H()), 1),
    (lambda L: read(L, k=None), 1),
    (lambda L: read(L, v=H(2 * P), c=C(v_codes=None)), 1),
    (lambda L: fused(L, k=H(2 * P, heads=1)), 1),
    (lambda L: fused(L, c=C(heads=1)), 1),
    (lambda L: fused(L, d=8), 1),
    (lambda L: fused(L, slots=None), 1),
    (lambda L: fused(L, eps=-1.0), 1),
    (lambda L: fused(L, qo=H(4 * P)), 1),
    (lambda L: fused(L, ko=H(4 * P)), 1),
    (lambda L: fused(L, ko=H()), 1),
    (lambda L: L.nrm_qk_norm_rope_cache(H(), None, H(4 * P), None, None, None, H(3 * P), None, C(), P, 8, 16, 1e-6, 1, 0,
                                        None), 1),
])
def test_bad_arguments_are_refused_on_the_host(lib, call, expect):
    assert call(lib) == expect
    assert nrm.nrm_last_error_message() != ""


def test_without_keys_their_arguments_are_ignored(lib):
    # (no tokens: nothing is enqueued on a GPU)
    odd = P + 1
    assert lib.nrm_qk_norm_rope_fwd(H(), None, None, odd, None, H(3 * P), None, None, odd, 0, 16, 1e-6, 0, None) != 1
    assert lib.nrm_qk_norm_rope_bwd(H(2 * P), None, H(), None, None, odd, P, odd, None, H(3 * P), None, None, None, 0, 16,
                                    0, None, 0, None) != 1
    with pytest.raises(ValueError, match="current CUDA device"):
        nrm.nrm_qk_norm_rope_fwd(**_qk(wk=torch.ones(3), rstd_k=torch.ones(5)))


def test_structures_match_the_header(tmp_path):
    import os
    import subprocess
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "libnorm.h"\nint main(void) { printf("%zu %zu %zu\\n", sizeof(nrm_heads), '
                   'sizeof(nrm_rope), sizeof(nrm_kv_cache)); return 0; }\n')
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-I", os.path.join(nbuild.ROOT, "include"), str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in out] == [ctypes.sizeof(t) for t in (B._Heads, B._Rope, B._Cache)]


# ---------------------------------------------------------------------------
# refusals of the binding (tensors on the CPU: shapes and types first, then the device)
# ---------------------------------------------------------------------------

def _qk(**k):
    a = dict(q=torch.zeros(4, 2, 16), k=None, wq=None, wk=None, pos=torch.arange(4), inv_freq=torch.ones(8),
             q_out=torch.zeros(4, 2, 16), k_out=None, rstd_q=None, rstd_k=None, eps=1e-6)
    a.update(k)
    return a


@pytest.mark.parametrize("change,error,text", [
    ({}, ValueError, "current CUDA device"),
    ({"q": torch.zeros(4, 32)}, ValueError, "must be"),
    ({"q": torch.zeros(4, 2, 32)[..., ::2]}, ValueError, "contiguous"),
    ({"q": torch.zeros(2, 8, 2, 16)[:, :2]}, ValueError, "one stride"),
    ({"q_out": torch.zeros(4, 3, 16)}, ValueError, "shape"),
    ({"q_out": torch.zeros(4, 2, 16).half()}, TypeError, "expected"),
    ({"k": torch.zeros(4, 1, 16)}, ValueError, "k_out"),
    ({"k": torch.zeros(3, 1, 16), "k_out": torch.zeros(3, 1, 16)}, ValueError, "tokens"),
    ({"wq": torch.ones(15)}, ValueError, "wq"),
    ({"wq": torch.ones(16).half()}, TypeError, "wq"),
    ({"rstd_q": torch.ones(7)}, ValueError, "rstd_q"),
    ({"rstd_q": torch.ones(8).double()}, TypeError, "rstd_q"),
    ({"pos": torch.arange(5)}, ValueError, "pos"),
    ({"pos": torch.arange(4).int()}, TypeError, "pos"),
    ({"pos": None}, TypeError, "pos"),
    ({"inv_freq": torch.ones(8).double()}, TypeError, "inv_freq"),
    ({"axis": bytes(7)}, ValueError, "pos|axis"),
    ({"axis": bytes(7), "pos": torch.zeros(2, 4, dtype=torch.int64)}, ValueError, "axis"),
    ({"pairs": "both"}, ValueError, "pairs"),
])
def test_binding_refuses(change, error, text):
    with pytest.raises(error, match=text):
        nrm.nrm_qk_norm_rope_fwd(**_qk(**change))


@pytest.mark.parametrize("codes,scales,error", [
    (torch.zeros(2, 4, 1, 16, dtype=torch.int16), torch.zeros(2, 4, 1, 1), TypeError),
    (torch.zeros(2, 4, 16, dtype=torch.int8), torch.zeros(2, 4, 1, 1), ValueError),
    (torch.zeros(2, 4, 1, 16, dtype=torch.int8), torch.zeros(2, 4, 1, 3), ValueError),
    (torch.zeros(2, 4, 1, 16, dtype=torch.int8), torch.zeros(2, 4, 2, 1), ValueError),
    (torch.zeros(2, 4, 1, 16, dtype=torch.int8), torch.zeros(2, 4, 1, 1).double(), ValueError),
    (torch.zeros(2, 4, 1, 32, dtype=torch.int8)[..., ::2], torch.zeros(2, 4, 1, 1), ValueError),
    (torch.zeros(2, 4, 1, 16, dtype=torch.int8), torch.zeros(2, 4, 1, 1), ValueError),  # on the CPU
])
def test_cache_handle_refuses(codes, scales, error):
    with pytest.raises(error):
        nrm.kv_cache(codes, scales)


def test_cache_handle_refuses_keys_and_values_that_differ():
    a, s = torch.zeros(2, 4, 1, 16, dtype=torch.int8), torch.zeros(2, 4, 1, 1)
    with pytest.raises(ValueError, match="strides"):
        nrm.kv_cache(a, s, torch.zeros(2, 1, 4, 16, dtype=torch.int8).transpose(1, 2), s)
    with pytest.raises(ValueError, match="together"):
        nrm.kv_cache(a, s, a, None)
