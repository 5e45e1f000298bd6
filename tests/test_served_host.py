"""Attention over the cache, eviction from it and the norms around a block without a GPU: the
reference against differences and closed forms, and every refusal of the C entry points and of
the binding (all before anything is enqueued)."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
from normalization_layernorm_rmsnorm_gb300 import _binding as B
from normalization_layernorm_rmsnorm_gb300 import build as nbuild
from oracle import heads
from oracle import served as ref
from test_dependent_launch import code, kernels
from test_heads_host import C, H, P


@pytest.fixture(scope="module")
def lib():
    nbuild.build()
    return nrm.load()


# ---------------------------------------------------------------------------
# the reference
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("gates,post,pre,stream", [(0, True, True, True), (1, True, True, True), (3, True, True, False),
                                                   (6, False, True, True), (2, True, False, True)])
def test_reference_block_gradients_against_differences(gates, post, pre, stream):
    rng = np.random.default_rng(gates)
    rows, cols, alpha, eps = 6, 5, 0.7, 1e-3
    v = {"x": rng.normal(size=(rows, cols)), "f": rng.normal(size=(rows, cols)), "w_post": 1 + 0.1 * rng.normal(size=cols),
         "w_pre": 1 + 0.1 * rng.normal(size=cols), "gate": rng.normal(size=(gates, cols)) if gates else None}
    dh = rng.normal(size=(rows, cols)) if pre else None
    dy = rng.normal(size=(rows, cols)) if stream else None

    def forward(x, f, w_post, w_pre, gate):
        y, r1 = ref.block_fwd(x, f, gate, w_post, alpha, eps, post)
        h, r2 = ref.block_pre(y, w_pre, eps)
        return y, h, r1, r2

    def loss(**a):
        y, h, _, _ = forward(**a)
        return (0 if dh is None else (dh * h).sum()) + (0 if dy is None else (dy * y).sum())

    y, h, r1, r2 = forward(**v)
    got = dict(zip(("x", "f", "gate", "w_post", "w_pre"),
                   ref.block_bwd(dh, dy, v["f"], y, v["gate"], v["w_post"], v["w_pre"], r1, r2, alpha, post)))
    step = 1e-6
    # central differences: truncation step^2 and rounding 1e-15 / step, both far below 1e-7
    for n, g in got.items():
        if g is None:
            continue
        for i in np.ndindex(v[n].shape):
            e = np.zeros_like(v[n])
            e[i] = step
            d = (loss(**{**v, n: v[n] + e}) - loss(**{**v, n: v[n] - e})) / (2 * step)
            assert abs(d - g[i]) < 1e-7, (n, i)


def test_reference_attention_closed_forms():
    k, v = np.zeros((3, 2, 1, 2)), np.arange(12.0).reshape(3, 2, 1, 2)
    table, q = np.array([[2, 0]]), np.ones((1, 3, 2))
    # equal logits: the mean of the values; pages in the table's order
    out, lse, w, _, _ = ref.attention(q, k, v, table, [3], 1.0)
    np.testing.assert_allclose(out[0], np.tile((v[2, 0, 0] + v[2, 1, 0] + v[0, 0, 0]) / 3, (3, 1)))
    np.testing.assert_allclose(lse, np.log(3))
    np.testing.assert_allclose(w[0, 0], [1, 1, 1, 0])  # three heads share it
    out, lse, w, _, _ = ref.attention(q, k, v, table, [3], 1.0, window=1)
    np.testing.assert_allclose(out[0, 0], v[0, 0, 0])
    np.testing.assert_allclose(w[0, 0], [0, 0, 3, 0])
    # a far larger logit takes all
    k[2, 1] = 500
    np.testing.assert_allclose(ref.attention(q, k, v, table, [3], 1.0)[0][0, 0], v[2, 1, 0])
    out, lse, _, _, _ = ref.attention(q, k, v, table, [0], 1.0)
    assert not out.any() and np.isneginf(lse).all()


def test_reference_stored_values_are_those_of_the_cache():
    rng = np.random.default_rng(0)
    for kind in ("e4m3", "int8", "int4"):
        codes, scales = heads.quantise(rng.normal(size=(3, 8)), kind, 4)
        held = codes if kind != "int4" else ((codes[..., 0::2].astype(int) & 15) | (codes[..., 1::2].astype(int) & 15) << 4)
        np.testing.assert_array_equal(ref.stored(held, scales, kind), codes * np.repeat(scales.astype(np.float64), 4, -1))


def test_reference_eviction_by_hand():
    w = np.array([[[5.0, 1.0, 7.0, 7.0, 0.0, 7.0, 2.0]]])
    kept, new = ref.evict(w, [7], 4, 1, 1, 8)
    # the first and the last stay; of three sevens the earlier two
    assert kept.tolist() == [[[0, 2, 3, 6]]] and new.tolist() == [4]
    assert ref.evict(w, [3], 4, 1, 1, 8)[0].tolist() == [[[0, 1, 2, -1]]]
    w[0, 0, 4] = np.nan
    assert ref.evict(w, [7], 2, 0, 0, 8)[0].tolist() == [[[2, 4]]]
    assert ref.evict(w, [7], 3, 2, 1, 8)[0].tolist() == [[[0, 1, 6]]]


# ---------------------------------------------------------------------------
# refusals of the C entry points
# ---------------------------------------------------------------------------

def G(table=P, lengths=P, sequences=8, width=4, stride=4):
    return B._Pages(table, lengths, sequences, width, stride)


def W(data=P, capacity=32, ss=64, hs=32):
    return B._Weights(data, capacity, ss, hs)


def attend(L, q=None, c=None, g=None, out=None, scale=1.0, window=0, lse=None, w=None, dt=0, ws=None, n=0):
    return L.nrm_kv_cache_attention(q or H(heads=4, ts=64), c or C(), g or G(), out or H(3 * P, heads=4, ts=64), scale, window,
                                    lse, w, dt, ws, n, None)


def evict(L, c=None, g=None, w=W(), table=2 * P, width=4, stride=4, lengths=2 * P, nw=None, kept=P, keep=16, first=0, recent=0):
    return L.nrm_kv_cache_evict(c or C(), g or G(), w, table, width, stride, lengths, nw, kept, keep, first, recent, None)


def block(L, x=P, f=2 * P, gate=None, w1=None, w2=None, y=3 * P, h=4 * P, r1=None, r2=None, rows=8, cols=16, gates=0, alpha=1.0,
          eps=1e-6, post=1, dt=0):
    return L.nrm_block_norm_fwd(x, f, gate, w1, w2, y, h, r1, r2, rows, cols, gates, alpha, eps, post, dt, None)


def block_bwd(L, dh=P, dy=2 * P, f=3 * P, y=4 * P, gate=None, w1=None, w2=None, r1=P, r2=P, dx=5 * P, df=6 * P, dg=None, dw1=None,
              dw2=None, rows=8, cols=16, gates=0, alpha=1.0, post=1, dt=0, ws=None, n=0):
    return L.nrm_block_norm_bwd(dh, dy, f, y, gate, w1, w2, r1, r2, dx, df, dg, dw1, dw2, rows, cols, gates, alpha, post, dt, ws, n,
                                None)


@pytest.mark.parametrize("call,expect", [
    (lambda L: attend(L, dt=3), 1),
    (lambda L: attend(L, q=H(heads=3, ts=64), out=H(3 * P, heads=3, ts=64)), 1),  # no multiple of the cache's heads
    (lambda L: attend(L, q=H(data=None, heads=4, ts=64)), 1),
    (lambda L: attend(L, out=H(3 * P, heads=2, ts=64)), 1),
    (lambda L: attend(L, out=H(heads=4, ts=64)), 1),  # in place
    (lambda L: attend(L, out=H(3 * P, heads=4, ts=63)), 1),
    (lambda L: attend(L, scale=float("inf")), 1),
    (lambda L: attend(L, scale=float("nan")), 1),
    (lambda L: attend(L, window=-1), 1),
    (lambda L: attend(L, lse=P + 2), 1),
    (lambda L: attend(L, c=C(v_codes=None)), 1),
    (lambda L: attend(L, c=C(group=5)), 1),
    (lambda L: L.nrm_kv_cache_attention(H(heads=4, ts=64), None, G(), H(3 * P, heads=4, ts=64), 1.0, 0, None, None, 0, None, 0, None), 1),
    (lambda L: L.nrm_kv_cache_attention(H(heads=4, ts=64), C(), None, H(3 * P, heads=4, ts=64), 1.0, 0, None, None, 0, None, 0, None), 1),
    (lambda L: attend(L, g=G(table=None)), 1),
    (lambda L: attend(L, g=G(table=P + 4)), 1),
    (lambda L: attend(L, g=G(lengths=None)), 1),
    (lambda L: attend(L, g=G(lengths=P + 4)), 1),
    (lambda L: attend(L, g=G(sequences=-1)), 1),
    (lambda L: attend(L, g=G(sequences=(1 << 30) + 1)), 2),
    (lambda L: attend(L, g=G(width=0)), 1),
    (lambda L: attend(L, g=G(stride=3)), 1),
    (lambda L: attend(L, g=G(width=1 << 38, stride=1 << 38)), 2),
    (lambda L: attend(L, w=W(data=None)), 1),
    (lambda L: attend(L, w=W(data=P + 2)), 1),
    (lambda L: attend(L, w=W(capacity=0)), 1),
    (lambda L: attend(L, w=W(hs=31)), 1),
    (lambda L: attend(L, w=W(ss=63)), 1),
    (lambda L: attend(L, w=W(hs=-32)), 1),
    (lambda L: evict(L, w=None), 1),
    (lambda L: evict(L, c=C(k_codes=None)), 1),
    (lambda L: evict(L, c=C(v_codes=P)), 1),
    (lambda L: evict(L, keep=0), 1),
    (lambda L: evict(L, keep=33), 1),  # more than the new pages hold
    (lambda L: evict(L, first=-1), 1),
    (lambda L: evict(L, recent=-1), 1),
    (lambda L: evict(L, first=9, recent=8), 1),
    (lambda L: evict(L, first=(1 << 62) + 5, recent=(1 << 62)), 1),
    (lambda L: evict(L, table=None), 1),
    (lambda L: evict(L, table=P), 1),
    (lambda L: evict(L, stride=3), 1),
    (lambda L: evict(L, lengths=None), 1),
    (lambda L: evict(L, lengths=P), 1),
    (lambda L: evict(L, lengths=2 * P + 4), 1),
    (lambda L: evict(L, kept=None), 1),
    (lambda L: evict(L, kept=P + 4), 1),
    (lambda L: evict(L, nw=W(data=2 * P, capacity=15)), 1),
    (lambda L: evict(L, nw=W()), 1),
    (lambda L: evict(L, nw=W(data=2 * P, hs=16)), 1),
    (lambda L: evict(L, g=G(lengths=None)), 1),
    (lambda L: evict(L, g=G(width=1 << 30, stride=1 << 30), w=W(capacity=1 << 33, hs=1 << 33, ss=1 << 34)), 2),
    (lambda L: block(L, dt=3), 1),
    (lambda L: block(L, rows=-1), 1),
    (lambda L: block(L, cols=0), 1),
    (lambda L: block(L, cols=(1 << 27) + 1), 2),
    (lambda L: block(L, rows=1 << 39), 2),
    (lambda L: block(L, eps=0.0), 1),
    (lambda L: block(L, alpha=float("nan")), 1),
    (lambda L: block(L, x=None), 1),
    (lambda L: block(L, f=None), 1),
    (lambda L: block(L, y=None), 1),
    (lambda L: block(L, x=P + 2), 1),
    (lambda L: block(L, gates=1), 1),
    (lambda L: block(L, gate=P), 1),
    (lambda L: block(L, gate=P, gates=3), 1),
    (lambda L: block(L, gate=P, gates=-1), 1),
    (lambda L: block(L, y=2 * P), 1),
    (lambda L: block(L, h=P), 1),
    (lambda L: block(L, h=3 * P), 1),
    (lambda L: block(L, r1=P, r2=P), 1),
    (lambda L: block(L, r1=P + 1), 1),
    (lambda L: block(L, w1=P + 1), 1),
    (lambda L: block_bwd(L, dh=None, dy=None), 1),
    (lambda L: block_bwd(L, f=None), 1),
    (lambda L: block_bwd(L, y=None), 1),
    (lambda L: block_bwd(L, dx=None), 1),
    (lambda L: block_bwd(L, df=None), 1),
    (lambda L: block_bwd(L, r1=None), 1),
    (lambda L: block_bwd(L, r2=None), 1),
    (lambda L: block_bwd(L, dx=P), 1),
    (lambda L: block_bwd(L, df=2 * P), 1),
    (lambda L: block_bwd(L, df=5 * P), 1),
    (lambda L: block_bwd(L, dw1=P, post=0), 1),
    (lambda L: block_bwd(L, dw2=P, dh=None), 1),
    (lambda L: block_bwd(L, dg=P), 1),
    (lambda L: block_bwd(L, dw1=P, dw2=P), 1),
    (lambda L: block_bwd(L, dw1=P, dg=P, gate=P, gates=2), 1),
    (lambda L: block_bwd(L, gate=P, gates=5), 1),
    (lambda L: block_bwd(L, alpha=float("inf")), 1),
    (lambda L: block_bwd(L, dx=5 * P + 2), 1),
    (lambda L: block_bwd(L, dt=-1), 1),
])
def test_bad_arguments_are_refused_on_the_host(lib, call, expect):
    assert call(lib) == expect
    assert nrm.nrm_last_error_message() != ""


def test_without_a_part_its_arguments_are_ignored(lib):
    # (no rows: nothing is enqueued on a GPU)
    odd = P + 1
    assert block(lib, w1=odd, r1=odd, post=0, rows=0) != 1
    assert block(lib, h=None, w2=odd, r2=odd, rows=0) != 1


def test_structures_match_the_header(tmp_path):
    src = tmp_path / "sizes.c"
    src.write_text('#include <stdio.h>\n#include "libnorm.h"\nint main(void) { printf("%zu %zu\\n", sizeof(nrm_kv_pages), '
                   'sizeof(nrm_kv_weights)); return 0; }\n')
    exe = str(tmp_path / "sizes")
    subprocess.run(["gcc", "-I", os.path.join(nbuild.ROOT, "include"), str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in out] == [ctypes.sizeof(t) for t in (B._Pages, B._Weights)]


# ---------------------------------------------------------------------------
# refusals of the binding (tensors on the CPU: shapes and types first, then the device)
# ---------------------------------------------------------------------------

class _Cache:
    """What the calls take of a cache handle."""

    def __init__(self):
        self.c = C()
        self.address, self.held = ctypes.addressof(self.c), torch.zeros(4, 8, 2, 16, dtype=torch.int8)


def _long(*shape):
    return torch.zeros(shape, dtype=torch.int64)


@pytest.mark.parametrize("change,error,text", [
    ({}, ValueError, "current CUDA device"),
    ({"q": torch.zeros(3, 64)}, ValueError, "must be"),
    ({"q": torch.zeros(3, 4, 8), "out": torch.zeros(3, 4, 8)}, ValueError, "rows of"),
    ({"out": torch.zeros(3, 4, 15)}, ValueError, "shape"),
    ({"out": torch.zeros(3, 4, 16).half()}, TypeError, "expected"),
    ({"table": _long(3)}, ValueError, "table"),
    ({"table": _long(3, 4).int()}, ValueError, "table"),
    ({"table": _long(2, 4)}, ValueError, "sequences"),
    ({"table": _long(4, 3).t()}, ValueError, "contiguous"),
    ({"lengths": _long(4)}, ValueError, "lengths"),
    ({"lengths": _long(3).int()}, TypeError, "lengths"),
    ({"lse": torch.zeros(3, 3)}, ValueError, "lse"),
    ({"lse": torch.zeros(3, 4).double()}, TypeError, "lse"),
    ({"weights": torch.zeros(3, 4, 32)}, ValueError, "weights"),
    ({"weights": torch.zeros(3, 2, 32).half()}, ValueError, "weights"),
    ({"weights": torch.zeros(3, 32, 2).transpose(1, 2)}, ValueError, "contiguous"),
    ({"workspace": torch.zeros(64)[::2]}, ValueError, "workspace"),
    ({"window": 1.5}, TypeError, "integer"),
    ({"scale": "1"}, TypeError, "real number"),
    ({"workspace": 3}, TypeError, "workspace"),
])
def test_attention_binding_refuses(change, error, text):
    a = dict(q=torch.zeros(3, 4, 16), cache=_Cache(), table=_long(3, 4), lengths=_long(3), out=torch.zeros(3, 4, 16), scale=1.0,
             workspace=torch.zeros(64))
    with pytest.raises(error, match=text):
        nrm.nrm_kv_cache_attention(**{**a, **change})


@pytest.mark.parametrize("change,error,text", [
    ({}, ValueError, "current CUDA device"),
    ({"table": _long(3)}, ValueError, "table"),
    ({"lengths": _long(2)}, ValueError, "lengths"),
    ({"weights": torch.zeros(3, 1, 32)}, ValueError, "weights"),
    ({"new_table": _long(2, 2)}, ValueError, "new_table"),
    ({"new_table": _long(3, 2).int()}, ValueError, "new_table"),
    ({"new_lengths": _long(2)}, ValueError, "new_lengths"),
    ({"new_weights": torch.zeros(3, 3, 9)}, ValueError, "new_weights"),
    ({"kept": _long(3, 9)}, ValueError, "kept"),
    ({"kept": _long(3, 3, 9)}, ValueError, "kept"),
    ({"kept": _long(3, 2, 9).int()}, TypeError, "kept"),
    ({"kept": _long(3, 9, 2).transpose(1, 2)}, ValueError, "kept"),
    ({"weights": None}, ValueError, "weights"),
])
def test_eviction_binding_refuses(change, error, text):
    a = dict(cache=_Cache(), table=_long(3, 4), lengths=_long(3), weights=torch.zeros(3, 2, 32), new_table=_long(3, 2),
             new_lengths=_long(3), new_weights=None, kept=_long(3, 2, 9))
    with pytest.raises(error, match=text):
        nrm.nrm_kv_cache_evict(**{**a, **change})


def _rows(**k):
    t = torch.zeros(6, 16)
    return {**dict(x=t, f=t, gate=None, w_post=None, w_pre=None, y=t, h=t, rstd_post=None, rstd_pre=None, alpha=1.0, eps=1e-6), **k}


@pytest.mark.parametrize("change,error,text", [
    ({}, ValueError, "current CUDA device"),
    ({"x": torch.tensor(1.0)}, ValueError, "cols"),
    ({"x": torch.zeros(6, 16).double()}, TypeError, "dtype"),
    ({"f": torch.zeros(5, 16)}, ValueError, "shape"),
    ({"f": torch.zeros(6, 16).half()}, TypeError, "expected"),
    ({"y": torch.zeros(16, 6).t()}, ValueError, "contiguous"),
    ({"h": torch.zeros(96)}, ValueError, "shape"),
    ({"gate": torch.zeros(15)}, ValueError, "gate"),
    ({"gate": torch.zeros(2, 16).half()}, TypeError, "gate"),
    ({"w_post": torch.zeros(15)}, ValueError, "w_post"),
    ({"w_pre": torch.zeros(16).half()}, TypeError, "w_pre"),
    ({"rstd_post": torch.zeros(5)}, ValueError, "rstd_post"),
    ({"rstd_pre": torch.zeros(6).half()}, TypeError, "rstd_pre"),
    ({"y": None}, ValueError, "y"),
])
def test_block_binding_refuses(change, error, text):
    with pytest.raises(error, match=text):
        nrm.nrm_block_norm_fwd(**_rows(**change))


@pytest.mark.parametrize("change,error,text", [
    ({}, ValueError, "current CUDA device"),
    ({"dgate": torch.zeros(3, 16)}, ValueError, "dgate"),
    ({"y": None}, ValueError, "y"),
    ({"rstd_post": None}, ValueError, "rstd_post"),
    ({"dw_post": torch.zeros(17)}, ValueError, "dw_post"),
    ({"dx": torch.zeros(6, 15)}, ValueError, "dx"),
    ({"workspace": torch.zeros(64)[::2]}, ValueError, "workspace"),
])
def test_block_backward_binding_refuses(change, error, text):
    t, r = torch.zeros(6, 16), torch.zeros(6)
    a = dict(dh=t, dy=t, f=t, y=t, gate=torch.zeros(2, 16), w_post=None, w_pre=None, rstd_post=r, rstd_pre=r, dx=t, df=t,
             dgate=torch.zeros(2, 16), dw_post=None, dw_pre=None, workspace=None, alpha=1.0)
    with pytest.raises(error, match=text):
        nrm.nrm_block_norm_bwd(**{**a, **change})


# ---------------------------------------------------------------------------
# the sources
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("name", ["kvattn.cuh", "kvevict.cu", "blocknorm.cuh"])
def test_kernels_wait_and_have_no_read_only_loads(name):
    # every kernel is launched while its predecessor runs: it waits for its end, and reads by ordinary loads
    text = code(name)
    found = 0
    for signature, body in kernels(text):
        found += 1
        assert "pdl_next()" in body, signature
    assert found
    assert re.findall(r"__ldg|\.nc\b|__restrict__|ld_stream_v4|ld_cached_v4|load_vec", text) == []
