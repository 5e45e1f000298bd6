"""The operators on attention heads through libnorm's public calls, against the
double-precision reference (oracle/heads.py).

Tolerances, derived before the first run.  u = 2^-24 is half a step of float32,
h that of the storage type.
  * r: a sum of d <= 256 positive squares in chains of at most 16 terms and 5
    more levels is off by 21 u; halved by the root, and with rsqrtf (2 ulp, 4 u)
    and the division, r is off by at most R = 16 u.
  * y: the products with r and w add 2 u.  A pair (a, b) is turned with cos and
    sin off by 3 u each (the angle's conversion to float32 in half turns, pi *
    2^-25, and 1 ulp of the function), and 2 u for the product and sum:
    |dy| <= (16 + 2 + 3 + 2 + 1) u (|a| + |b|) = 24 u (|a| + |b|), then h |y|.
  * dx = r g - x f, f = r^3 s / d: g off by 6 u G, G = (|dy_a| + |dy_b|) |w| of
    its pair; with the saved r, |d(r g)| <= 24 u r G.  s is off by (21 + 6) u
    sum G|x|, r^3 by 48 u, and 5 products: |d(x f)| <= 80 u |x| r^3/d sum G|x|.
    Then h |dx|.
  * dw: terms G' |x| r (G' without w) off by 24 u, and added in a chain of at
    most rows / 2 terms in a lane and 40 after it (two rows at least go to other
    lanes or warps): (64 + rows / 2) u sum G'|x| r, then h |dw|.
Codes, scales and values of the cache are whole roundings: equal, bit for bit.
"""
import numpy as np
import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
from oracle import heads as ref
from test_robustness import Guarded

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}  # half a step of the smallest numbers
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "int4": torch.uint8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    nrm.load()


def half_step(dtype):
    return torch.finfo(DT[dtype]).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def bits(t):
    return t.contiguous().view(torch.uint8)


def same(a, b):
    return torch.equal(bits(a), bits(b))


def within(got, want, err32, dtype, what):
    """|got - want| <= err32, and half a step of the storage type."""
    got, want = f64(got) if isinstance(got, torch.Tensor) else got, np.asarray(want)
    assert got.shape == want.shape, what
    lim = err32 + half_step(dtype) * (np.abs(want) + err32) * (dtype != "f32") + TINY[dtype]
    bad = ~(np.abs(got - want) <= lim)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off; worst {np.abs(got - want)[bad].max():.3e} "
                           f"at {np.argwhere(bad)[0]}: got {got[bad][0]!r}, want {want[bad][0]!r}")


class Data:
    """Seeded inputs of one case; q, k, v sliced out of one projection, or tensors of their own."""

    def __init__(self, dtype, tokens, hq, hk, d, rot, axes=1, fused=False, offset=0, seed=0, far=0):
        g = torch.Generator().manual_seed(1000 * tokens + 10 * d + seed)
        self.dtype, self.tokens, self.hq, self.hk, self.d, self.rot = dtype, tokens, hq, hk, d, rot
        dt = DT[dtype]

        def rows(heads, loud=False):
            x = torch.randn(tokens, heads, d, generator=g)
            if loud:
                x[..., d // 3] *= 8
            return x

        q, k, v = rows(hq), rows(hk, True), rows(hk)
        if fused:
            qkv = torch.cat([q, k, v], 1).to(dt).cuda()
            self.q, self.k, self.v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        else:
            self.q, self.k, self.v = (self.place(x.to(dt), offset) for x in (q, k, v))
        self.dqo, self.dko = (self.place(rows(n).to(dt), offset) for n in (hq, hk))
        self.wq, self.wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(dt).cuda() for _ in range(2))
        self.pos = torch.randint(0, 5000, (axes, tokens), generator=g).cuda() + far
        self.inv = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(rot // 2, 1))).float().cuda()
        self.axis = bytes(p % axes for p in range(rot // 2)) if axes > 1 else None
        if rot == 0:
            self.pos = self.inv = self.axis = None

    @staticmethod
    def place(x, offset):
        """x on the GPU, `offset` elements into its buffer."""
        b = torch.empty(x.numel() + offset, dtype=x.dtype, device="cuda")
        v = b[offset:].view(x.shape)
        v.copy_(x)
        return v

    def angles(self):
        if self.rot == 0:
            return np.zeros((self.tokens, 0))
        return ref.angles(self.pos.cpu().numpy(), self.inv.cpu().numpy(), self.axis)


LAYOUTS = [
    # dtype, tokens, hq, hk, d, rot, pairs, axes, fused, offset (elements off 16 bytes)
    ("bf16", 1, 32, 8, 128, 128, "half", 1, False, 0),
    ("bf16", 33, 4, 2, 128, 128, "half", 1, True, 0),
    ("f16", 17, 6, 3, 64, 64, "pair", 2, True, 0),
    ("f16", 5, 3, 1, 256, 64, "pair", 1, False, 0),
    ("f32", 19, 5, 5, 80, 40, "half", 3, True, 0),
    ("f32", 7, 2, 1, 256, 256, "half", 1, False, 0),
    ("bf16", 9, 3, 3, 96, 32, "half", 3, False, 0),
    ("bf16", 300, 2, 1, 64, 32, "half", 1, True, 0),
    ("bf16", 11, 2, 2, 72, 72, "half", 2, False, 0),
    ("f16", 13, 3, 1, 40, 10, "pair", 1, True, 0),
    ("f32", 3, 2, 1, 8, 4, "half", 1, False, 0),
    ("bf16", 6, 3, 2, 128, 128, "pair", 4, False, 1),
    ("f16", 21, 1, 1, 33, 16, "half", 1, False, 0),
    ("f32", 4, 1, 2, 1, 0, "half", 1, False, 0),
    ("bf16", 8, 2, 2, 2, 2, "half", 1, False, 0),
    ("bf16", 10, 4, 1, 160, 0, "half", 1, True, 0),
    ("f32", 6, 2, 2, 255, 254, "pair", 1, False, 0),
    ("f16", 4, 2, 1, 255, 254, "half", 4, False, 1),
    ("bf16", 5, 2, 2, 72, 36, "half", 1, False, 4),
    ("f32", 12, 3, 1, 36, 36, "pair", 1, False, 2),
    ("bf16", 700, 9, 2, 128, 128, "half", 1, False, 0),
    ("f16", 15, 3, 1, 72, 20, "pair", 3, False, 0),
    ("bf16", 8, 2, 2, 128, 124, "half", 1, False, 2),
    ("f16", 40, 12, 1, 40, 20, "half", 1, True, 0),
    ("bf16", 2000, 3, 1, 64, 64, "pair", 2, False, 0),
    # few heads of many tokens: several tokens share a warp's rows
    ("bf16", 20001, 1, 1, 16, 8, "half", 2, False, 0),
    ("f16", 5003, 2, 1, 64, 64, "pair", 1, True, 0),
    ("f32", 2503, 1, 2, 128, 64, "half", 3, False, 0),
]


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("dtype,tokens,hq,hk,d,rot,pairs,axes,fused,offset", LAYOUTS)
def test_norm_rope_forward_and_backward(dtype, tokens, hq, hk, d, rot, pairs, axes, fused, offset, weights):
    c = Data(dtype, tokens, hq, hk, d, rot, axes, fused, offset)
    eps = 1e-5
    wq, wk = (c.wq, c.wk) if weights else (None, None)
    dt = DT[dtype]
    out = {n: Guarded((tokens, h, d), dt, offset * c.q.element_size())
           for n, h in (("qo", hq), ("ko", hk), ("dq", hq), ("dk", hk))}
    out |= {"rq": Guarded((tokens, hq), torch.float32), "rk": Guarded((tokens, hk), torch.float32),
            "dwq": Guarded((d,), dt), "dwk": Guarded((d,), dt)}
    ws = Guarded((nrm.nrm_workspace_bytes(nrm.NRM_OP_QK_NORM_BWD, tokens, d, nrm.NRM_F32),), torch.uint8)
    o = {n: g.t for n, g in out.items()}
    how = dict(axis=c.axis, pairs=pairs)

    def both():
        nrm.nrm_qk_norm_rope_fwd(c.q, c.k, wq, wk, c.pos, c.inv, o["qo"], o["ko"], o["rq"], o["rk"], eps, **how)
        nrm.nrm_qk_norm_rope_bwd(c.dqo, c.dko, c.q, c.k, wq, wk, o["rq"], o["rk"], c.pos, c.inv, o["dq"], o["dk"],
                                 o["dwq"], o["dwk"], ws.t, **how)
        nrm.nrm_sync_status()

    both()
    for n, g in list(out.items()) + [("workspace", ws)]:
        g.check(n)
    first = {n: t.clone() for n, t in o.items()}
    for t in o.values():
        t.zero_()
    ws.t.fill_(0xFF)
    both()
    for n in o:
        assert same(first[n], o[n]), f"{n} differs between runs"

    ang = c.angles()
    n2 = rot // 2
    for x, w, dy, y, r, dx, dw, tag in ((c.q, wq, c.dqo, o["qo"], o["rq"], o["dq"], o["dwq"], "q"),
                                        (c.k, wk, c.dko, o["ko"], o["rk"], o["dk"], o["dwk"], "k")):
        x, dy, w = f64(x), f64(dy), None if w is None else f64(w)
        want, rr = ref.norm_rope_fwd(x, w, ang, eps, pairs)
        within(r, rr, 16 * U * rr, "f32", f"rstd_{tag}")
        normed = x * rr[..., None] * (1.0 if w is None else w)
        within(y, want, 24 * U * ref.pair_size(normed, n2, pairs), dtype, f"{tag}_out")
        wdx, wdw = ref.norm_rope_bwd(dy, x, w, ang, eps, pairs)
        gp = ref.pair_size(dy, n2, pairs)
        gw = gp * (1.0 if w is None else np.abs(w))
        r3 = rr[..., None]
        e = 24 * U * r3 * gw + 80 * U * np.abs(x) * r3 ** 3 * (gw * np.abs(x)).mean(-1, keepdims=True)
        within(dx, wdx, e, dtype, f"d{tag}")
        e = (64 + x.shape[0] * x.shape[1] / 2) * U * (gp * np.abs(x) * r3).sum((0, 1))
        within(dw, wdw, e, dtype, f"dw{tag}")


def test_gradients_against_differences():
    # <dx, v> against a central difference of the double-precision forward along v:
    # dx is off by what the bound of dx allows, its rounding to float32 among it
    c = Data("f32", 5, 3, 2, 64, 32)
    rq, rk = torch.empty(5, 3, device="cuda"), torch.empty(5, 2, device="cuda")
    qo, ko, dq, dk = (torch.empty_like(t) for t in (c.q, c.k, c.q, c.k))
    dwq, dwk = torch.empty_like(c.wq), torch.empty_like(c.wk)
    nrm.nrm_qk_norm_rope_fwd(c.q, c.k, c.wq, c.wk, c.pos, c.inv, qo, ko, rq, rk, 1e-6)
    nrm.nrm_qk_norm_rope_bwd(c.dqo, c.dko, c.q, c.k, c.wq, c.wk, rq, rk, c.pos, c.inv, dq, dk, dwq, dwk,
                             nrm.qk_norm_workspace(c.q))
    ang = c.angles()
    rng = np.random.default_rng(1)
    for x, w, dy, dx, dw in ((c.q, c.wq, c.dqo, dq, dwq), (c.k, c.wk, c.dko, dk, dwk)):
        x, w, dy = f64(x), f64(w), f64(dy)
        vx, vw, h = rng.normal(size=x.shape), rng.normal(size=w.shape), 1e-5

        def loss(s):
            return (ref.norm_rope_fwd(x + s * vx, w + s * vw, ang, 1e-6)[0] * dy).sum()

        want = (loss(h) - loss(-h)) / (2 * h)
        got = (f64(dx) * vx).sum() + (f64(dw) * vw).sum()
        # |dx - exact| <= (24 + 80 + 1) u * size and |dw - exact| <= 80 u * size, size the terms' absolute sum
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True))
        g = ref.pair_size(dy, 16) * np.abs(w)
        size = ((r * g + np.abs(x) * r ** 3 * (g * np.abs(x)).mean(-1, keepdims=True)) * np.abs(vx)).sum()
        size += ((ref.pair_size(dy, 16) * np.abs(x) * r).sum((0, 1)) * np.abs(vw)).sum()
        assert abs(got - want) <= 105 * U * size + 1e-8 * abs(want)


@pytest.mark.parametrize("dtype,tokens,hq,hk,d,rot,pairs,axes,fused,offset", LAYOUTS)
def test_rope_forward_backward_and_in_place(dtype, tokens, hq, hk, d, rot, pairs, axes, fused, offset):
    c = Data(dtype, tokens, hq, hk, d, rot, axes, fused, offset, seed=1)
    how = dict(axis=c.axis, pairs=pairs)
    qo, ko, dq, dk = (Guarded(t.shape, t.dtype, offset * t.element_size()) for t in (c.q, c.k, c.q, c.k))
    nrm.nrm_rope_fwd(c.q, c.k, c.pos, c.inv, qo.t, ko.t, **how)
    nrm.nrm_rope_bwd(c.dqo, c.dko, c.pos, c.inv, dq.t, dk.t, **how)
    nrm.nrm_sync_status()
    ang = c.angles()
    for g, x, inverse, tag in ((qo, c.q, False, "q_out"), (ko, c.k, False, "k_out"), (dq, c.dqo, True, "dq"),
                               (dk, c.dko, True, "dk")):
        g.check(tag)
        want = ref.rotate(f64(x), ang, pairs, inverse)
        within(g.t, want, 8 * U * ref.pair_size(f64(x), rot // 2, pairs), dtype, tag)
    # in place gives the same bits
    q, k = c.q.clone(), c.k.clone()
    nrm.nrm_rope_fwd(q, k, c.pos, c.inv, q, k, **how)
    assert same(q, qo.t) and same(k, ko.t)


def test_norm_rope_in_place_inside_a_fused_projection():
    c = Data("bf16", 40, 4, 2, 128, 128, fused=True)
    qo, ko = torch.empty(40, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(40, 2, 128, dtype=torch.bfloat16,
                                                                                     device="cuda")
    nrm.nrm_qk_norm_rope_fwd(c.q, c.k, c.wq, c.wk, c.pos, c.inv, qo, ko, None, None, 1e-6)
    v = c.v.clone()
    nrm.nrm_qk_norm_rope_fwd(c.q, c.k, c.wq, c.wk, c.pos, c.inv, c.q, c.k, None, None, 1e-6)
    assert same(c.q, qo) and same(c.k, ko) and same(c.v, v)


def test_queries_alone_and_batched_views():
    c = Data("f16", 24, 4, 2, 64, 64)
    want = torch.empty_like(c.q)
    other = torch.empty_like(c.k)
    nrm.nrm_qk_norm_rope_fwd(c.q, c.k, c.wq, c.wk, c.pos, c.inv, want, other, None, None, 1e-6)
    got = torch.empty_like(c.q)
    nrm.nrm_qk_norm_rope_fwd(c.q, None, c.wq, None, c.pos, c.inv, got, None, None, None, 1e-6)
    assert same(got, want)
    # [batch, tokens, heads, d], and heads before tokens in memory
    got = torch.empty_like(c.q)
    nrm.nrm_qk_norm_rope_fwd(c.q.view(3, 8, 4, 64), None, c.wq, None, c.pos.view(3, 8), c.inv, got.view(3, 8, 4, 64), None,
                             None, None, 1e-6)
    assert same(got, want)
    t = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty(4, 24, 64, dtype=torch.float16, device="cuda").transpose(0, 1)
    nrm.nrm_qk_norm_rope_fwd(t, None, c.wq, None, c.pos, c.inv, out, None, None, None, 1e-6)
    assert same(out, want)
    # one row of frequencies seen by every token and head: an input expanded with zero strides
    row = c.q[:1, :1].expand(24, 4, 64)
    a, b = torch.empty_like(c.q), torch.empty_like(c.q)
    nrm.nrm_rope_fwd(row, None, c.pos, c.inv, a, None)
    nrm.nrm_rope_fwd(row.contiguous(), None, c.pos, c.inv, b, None)
    assert same(a, b)


@pytest.mark.parametrize("far", [0, 1 << 20, 1 << 31, -(1 << 33)])
def test_far_positions_keep_their_angles(far):
    # the input (1, 0) turned: cos and sin themselves.  Off by 3 u, and by 2 pi (|pos| 2^-52 + 2^-32) of the angle
    c = Data("f32", 50, 1, 1, 16, 16, far=far)
    q = torch.zeros(50, 1, 16, device="cuda")
    q[..., :8] = 1
    out = torch.empty_like(q)
    nrm.nrm_rope_fwd(q, None, c.pos, c.inv, out, None)
    a = c.angles()
    want = np.concatenate([np.cos(a), np.sin(a)], 1)[:, None]
    lim = 3 * U + 2 * np.pi * (abs(far) + 5000) * 2.0 ** -52 + 2 * np.pi * 2.0 ** -32 + 1e-15
    assert np.abs(f64(out) - want).max() <= lim


@pytest.mark.parametrize("scale", [0.0, 1e-30, 1e15])
def test_rows_of_zeros_and_of_extreme_size(scale):
    c = Data("f32", 6, 2, 1, 128, 64)
    q, k = c.q * scale, c.k * scale
    qo, ko, dq, dk = (torch.empty_like(t) for t in (q, k, q, k))
    rq, rk = torch.empty(6, 2, device="cuda"), torch.empty(6, 1, device="cuda")
    nrm.nrm_qk_norm_rope_fwd(q, k, c.wq, c.wk, c.pos, c.inv, qo, ko, rq, rk, 1e-6)
    nrm.nrm_qk_norm_rope_bwd(c.dqo, c.dko, q, k, c.wq, c.wk, rq, rk, c.pos, c.inv, dq, dk, None, None, None)
    x, ang = f64(q), c.angles()
    want, rr = ref.norm_rope_fwd(x, f64(c.wq), ang, 1e-6)
    within(rq, rr, 16 * U * rr, "f32", "rstd")
    within(qo, want, 24 * U * ref.pair_size(x * rr[..., None] * f64(c.wq), 32), "f32", "q_out")
    wdx, _ = ref.norm_rope_bwd(f64(c.dqo), x, f64(c.wq), ang, 1e-6)
    gw = ref.pair_size(f64(c.dqo), 32) * np.abs(f64(c.wq))
    r3 = rr[..., None]
    e = 24 * U * r3 * gw + 80 * U * np.abs(x) * r3 ** 3 * (gw * np.abs(x)).mean(-1, keepdims=True)
    within(dq, wdx, e + 1e-37, "f32", "dq")


def test_a_nan_stays_in_its_row():
    c = Data("bf16", 12, 3, 1, 128, 64)
    want, got = torch.empty_like(c.q), torch.empty_like(c.q)
    nrm.nrm_qk_norm_rope_fwd(c.q, None, c.wq, None, c.pos, c.inv, want, None, None, None, 1e-6)
    q = c.q.clone()
    q[4, 1, 7] = float("nan")
    q[7, 2, 100] = float("inf")
    nrm.nrm_qk_norm_rope_fwd(q, None, c.wq, None, c.pos, c.inv, got, None, None, None, 1e-6)
    assert got[4, 1].isnan().all()
    keep = torch.ones(12, 3, dtype=torch.bool, device="cuda")
    keep[4, 1] = keep[7, 2] = False
    assert same(got[keep], want[keep])
    # the rotation alone: only the pair of the NaN, and an infinity past the rotated part stays one
    q = c.q.clone()
    q[4, 1, 7] = float("nan")
    q[7, 2, 100] = float("inf")
    nrm.nrm_rope_fwd(q, None, c.pos, c.inv, got, None)
    assert int(got.isnan().sum()) == 2 and got[4, 1, 7].isnan() and got[4, 1, 39].isnan() and got[7, 2, 100].isinf()


def test_no_tokens():
    c = Data("bf16", 0, 2, 1, 64, 64)
    rq, rk = torch.empty(0, 2, device="cuda"), torch.empty(0, 1, device="cuda")
    dwq, dwk = torch.ones_like(c.wq), torch.ones_like(c.wk)
    nrm.nrm_qk_norm_rope_fwd(c.q, c.k, c.wq, c.wk, c.pos, c.inv, c.q, c.k, rq, rk, 1e-6)
    nrm.nrm_qk_norm_rope_bwd(c.dqo, c.dko, c.q, c.k, c.wq, c.wk, rq, rk, c.pos, c.inv, c.q, c.k, dwq, dwk,
                             nrm.qk_norm_workspace(c.q))
    cache = make_cache("int8", 2, 4, 1, 64, 64)
    slots = torch.empty(0, dtype=torch.int64, device="cuda")
    nrm.nrm_kv_cache_write(c.k, c.v, cache, slots)
    nrm.nrm_kv_cache_read(cache, slots, c.k, c.v)
    nrm.nrm_sync_status()
    assert not dwq.any() and not dwk.any()


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------

def make_cache(kind, pages, page, heads, d, group, layout="token", seed=0):
    """A cache full of noise.  layout: rows of a token together, or of a head ("head"), or keys
    and values in one buffer ("joined")."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    width = d // 2 if kind == "int4" else d

    def codes(shape):
        b = torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.int32)
        return b.to(torch.uint8).view(CODES[kind])

    def scales(shape):
        return torch.rand(shape, generator=g, device="cuda")

    if layout == "joined":
        c, s = codes((pages, 2, page, heads, width)), scales((pages, 2, page, heads, d // group))
        return nrm.kv_cache(c[:, 0], s[:, 0], c[:, 1], s[:, 1])
    if layout == "head":
        c = [codes((pages, heads, page, width)).transpose(1, 2) for _ in range(2)]
        s = [scales((pages, heads, page, d // group)).transpose(1, 2) for _ in range(2)]
    else:
        c = [codes((pages, page, heads, width)) for _ in range(2)]
        s = [scales((pages, page, heads, d // group)) for _ in range(2)]
    return nrm.kv_cache(c[0], s[0], c[1], s[1])


def numbers(codes, kind):
    """Codes as the numbers they are, in float64 (numpy)."""
    if kind == "int4":
        b = codes.cpu().numpy().astype(np.int64)
        n = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)
        return (n - 16 * (n > 7)).astype(np.float64)
    return codes.float().double().cpu().numpy()


def at_slots(t, slots):
    page = t.shape[1]
    raw = t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t
    return raw[slots // page, slots % page].view(t.dtype)


CACHES = [
    # dtype, kind, tokens, heads, d, group, page, layout, fused, offset
    ("bf16", "e4m3", 37, 8, 128, 128, 16, "token", False, 0),
    ("bf16", "int4", 65, 8, 128, 32, 16, "token", True, 0),
    ("f16", "int8", 50, 3, 64, 64, 8, "head", False, 0),
    ("f16", "int4", 33, 2, 256, 64, 100, "joined", False, 0),
    ("f16", "e4m3", 21, 3, 80, 40, 5, "token", True, 0),
    ("f32", "int8", 20, 2, 256, 256, 16, "token", False, 0),
    ("f32", "e4m3", 20, 1, 128, 16, 16, "joined", False, 0),
    ("f32", "int4", 9, 5, 64, 8, 7, "head", False, 0),
    ("bf16", "int8", 11, 2, 72, 24, 4, "token", False, 0),
    ("bf16", "e4m3", 11, 2, 96, 96, 4, "token", True, 1),
    ("f16", "int8", 5, 1, 33, 11, 3, "token", False, 0),
    ("f16", "int8", 5, 2, 7, 1, 3, "token", False, 1),
    ("f32", "int4", 5, 2, 30, 6, 3, "head", False, 0),
    ("bf16", "int8", 1, 1, 1, 1, 1, "token", False, 0),
    ("bf16", "int4", 1, 1, 2, 2, 1, "token", False, 0),
    ("f32", "int8", 3000, 2, 128, 64, 64, "token", False, 0),
    ("f32", "e4m3", 6, 2, 240, 80, 16, "token", False, 0),
    ("f32", "int4", 6, 2, 256, 32, 16, "token", False, 0),
    ("bf16", "int8", 14, 3, 160, 32, 16, "token", True, 0),
    ("bf16", "int4", 14, 3, 24, 8, 16, "token", False, 0),
    ("f16", "e4m3", 14, 3, 36, 12, 16, "token", False, 0),
    ("bf16", "int8", 14, 2, 128, 4, 16, "head", False, 2),
    ("f16", "int4", 14, 2, 128, 2, 16, "token", False, 2),
    ("f16", "int4", 9, 2, 44, 44, 16, "token", False, 0),
]


@pytest.mark.parametrize("dtype,kind,tokens,heads,d,group,page,layout,fused,offset", CACHES)
def test_cache_write_and_read(dtype, kind, tokens, heads, d, group, page, layout, fused, offset):
    c = Data(dtype, tokens, heads, heads, d, 0, fused=fused, offset=offset)
    pages = -(-tokens // page) + 2
    cache = make_cache(kind, pages, page, heads, d, group, layout)
    before = {n: getattr(cache, n).clone() for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
    g = torch.Generator().manual_seed(tokens)
    slots = torch.randperm(pages * page, generator=g)[:tokens].cuda()
    if tokens > 2:
        slots[tokens // 2] = -1  # a padded token
    k = c.k.clone() if not fused else c.k  # a few special rows: zeros, ties, a NaN, an infinity
    if tokens > 8:
        k[0] = 0
        k[1] = torch.arange(d, device="cuda").remainder(16).to(k.dtype) - 8
        k[2, 0, d // 2] = float("nan")
        k[3, 0, 0] = float("-inf")
        k[4] *= 1e-3
    nrm.nrm_kv_cache_write(k, c.v, cache, slots)
    nrm.nrm_sync_status()

    live = slots >= 0
    for x, codes, scales, n in ((k, cache.k_codes, cache.k_scales, "k"), (c.v, cache.v_codes, cache.v_scales, "v")):
        got_c, got_s = numbers(at_slots(codes, slots[live]), kind), at_slots(scales, slots[live]).cpu().numpy()
        x = f64(x[live])
        want_c, want_s = ref.quantise(x, kind, group)
        np.testing.assert_array_equal(np.isnan(got_s), np.isnan(want_s))
        np.testing.assert_array_equal(np.nan_to_num(got_s), np.nan_to_num(want_s), err_msg=f"{n} scales")
        if dtype == "f32":
            # the product x*q and the quotient are rounded: a value within 2 u of a border may go either way
            u = np.abs(x.reshape(*x.shape[:-1], -1, group) / np.where(want_s > 0, want_s, 1)[..., None].astype(np.float64))
            u = np.nan_to_num(u).reshape(x.shape)
            step = np.where(kind == "e4m3", 2.0 ** (np.floor(np.log2(np.maximum(u, 2.0 ** -6))) - 3), 1.0)
            near = np.abs(np.abs(want_c) - u) >= 0.5 * step - 8 * U * u
            np.testing.assert_array_equal(got_c[~near], want_c[~near], err_msg=f"{n} codes")
            assert (np.abs(got_c - want_c) <= step)[near].all() and near.mean() < 0.05
        else:
            np.testing.assert_array_equal(got_c, want_c, err_msg=f"{n} codes")
        # every other slot of the cache is as it was
        rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
        rest[slots[live]] = False
        where = torch.arange(pages * page, device="cuda")[rest]
        assert same(at_slots(codes.view(torch.uint8), where), at_slots(before[n + "_codes"].view(torch.uint8), where))
        assert same(at_slots(scales, where), at_slots(before[n + "_scales"], where))

    # read back, in another order and with repeats
    order = torch.randint(0, tokens, (tokens + 3,), generator=g).cuda()
    outs = {}
    for n in ("k", "v"):
        o = Guarded((tokens + 3, heads, d), DT[dtype], offset * c.k.element_size())
        o.t.fill_(7)
        outs[n] = o
    nrm.nrm_kv_cache_read(cache, slots[order], outs["k"].t, outs["v"].t)
    nrm.nrm_sync_status()
    left = slots[order] < 0
    for n, codes, scales in (("k", cache.k_codes, cache.k_scales), ("v", cache.v_codes, cache.v_scales)):
        outs[n].check(n)
        got = outs[n].t
        assert (got[left] == 7).all()
        src = slots[order][~left]
        num = torch.from_numpy(numbers(at_slots(codes, src), kind)).float()
        val = (num.unflatten(-1, (-1, group)) * at_slots(scales, src).cpu()[..., None]).flatten(-2).to(DT[dtype])
        got = got[~left].cpu()
        assert torch.equal(got.isnan(), val.isnan())
        assert torch.equal(got.nan_to_num(), val.nan_to_num())


def test_cache_keys_or_values_alone():
    c = Data("bf16", 12, 2, 2, 64, 0)
    full, part = make_cache("int8", 3, 8, 2, 64, 32), make_cache("int8", 3, 8, 2, 64, 32)
    slots = torch.arange(12, device="cuda")
    nrm.nrm_kv_cache_write(c.k, c.v, full, slots)
    nrm.nrm_kv_cache_write(c.k, None, part, slots)
    nrm.nrm_kv_cache_write(None, c.v, part, slots)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert same(getattr(full, n), getattr(part, n))
    only = nrm.kv_cache(full.k_codes, full.k_scales)
    a, b, v = torch.empty_like(c.k), torch.empty_like(c.k), torch.empty_like(c.v)
    nrm.nrm_kv_cache_read(full, slots, a, v)
    nrm.nrm_kv_cache_read(only, slots, b, None)
    assert same(a, b)
    nrm.nrm_kv_cache_read(full, slots, None, b)
    assert same(v, b)
    with pytest.raises(nrm.NrmError, match="no values"):
        nrm.nrm_kv_cache_write(c.k, c.v, only, slots)


def test_every_code_reads_back():
    # all 256 bytes as codes: e4m3 (its two NaNs among them) and whole numbers, and both halves of a byte
    byte = torch.arange(256, dtype=torch.int32, device="cuda").to(torch.uint8)
    slots = torch.zeros(1, dtype=torch.int64, device="cuda")
    scale = torch.full((1, 1, 1, 1), 0.75, device="cuda")
    for dtype in DT.values():
        out = torch.empty(1, 1, 256, dtype=dtype, device="cuda")
        for kind in ("e4m3", "int8"):
            codes = byte.view(CODES[kind]).view(1, 1, 1, 256)
            nrm.nrm_kv_cache_read(nrm.kv_cache(codes, scale), slots, out, None)
            want = (codes.cpu().float() * 0.75).to(dtype).view(-1)
            got = out.cpu().view(-1)
            assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())
        for part in (byte[:128], byte[128:]):
            nrm.nrm_kv_cache_read(nrm.kv_cache(part.view(1, 1, 1, 128), scale), slots, out, None)
            want = torch.from_numpy(numbers(part, "int4")).mul(0.75).to(dtype)
            assert torch.equal(out.cpu().view(-1), want)


@pytest.mark.parametrize("size", [1e-38, 2.0 ** -101, 2.0 ** -100, 1e-20, 1e20, 2.0 ** 101, 3e38])
@pytest.mark.parametrize("kind", ["e4m3", "int8", "int4"])
def test_groups_of_extreme_size(kind, size):
    x = torch.tensor([1.0, -0.5, 0.25, 0.1] * 8).mul(size).view(1, 1, 32).cuda()
    for dtype in ("f32", "bf16"):
        k = x.to(DT[dtype])
        cache = make_cache(kind, 1, 1, 1, 32, 32)
        nrm.nrm_kv_cache_write(k, None, cache, torch.zeros(1, dtype=torch.int64, device="cuda"))
        want_c, want_s = ref.quantise(f64(k), kind, 32)
        np.testing.assert_array_equal(numbers(cache.k_codes[0, 0], kind), want_c[0])
        np.testing.assert_array_equal(cache.k_scales.cpu().numpy().ravel(), want_s.ravel())


def test_slots_outside_the_cache_are_skipped_and_reported():
    c = Data("bf16", 6, 2, 2, 128, 128)
    cache = make_cache("int8", 2, 4, 2, 128, 128)
    before = cache.k_codes.clone(), cache.v_scales.clone()
    bad = torch.tensor([8, -2, 1 << 60, -(1 << 60), 2 ** 31, 100], device="cuda")
    nrm.nrm_kv_cache_write(c.k, c.v, cache, bad)
    with pytest.raises(nrm.NrmError) as e:
        nrm.nrm_sync_status()
    assert e.value.status == nrm.NRM_ERR_INVALID_ARG
    nrm.nrm_sync_status()  # the report is cleared
    assert same(before[0], cache.k_codes) and same(before[1], cache.v_scales)
    out = torch.full_like(c.k, 3)
    nrm.nrm_kv_cache_read(cache, bad, out, None)
    with pytest.raises(nrm.NrmError):
        nrm.nrm_sync_status()
    assert (out == 3).all()
    qo = torch.empty_like(c.q)
    nrm.nrm_qk_norm_rope_cache(c.q, c.k, c.v, c.wq, c.wk, c.pos, c.inv, qo, None, cache, bad, 1e-6)
    with pytest.raises(nrm.NrmError):
        nrm.nrm_sync_status()
    assert same(before[0], cache.k_codes) and same(before[1], cache.v_scales)
    # padding is not an error
    nrm.nrm_kv_cache_write(c.k, c.v, cache, torch.full_like(bad, -1))
    nrm.nrm_sync_status()


# ---------------------------------------------------------------------------
# together, as a served model uses them
# ---------------------------------------------------------------------------

SERVED = [
    # dtype, tokens, hq, hk, d, rot, pairs, axes, fused, offset, kind, group, page, layout
    ("bf16", 1, 32, 8, 128, 128, "half", 1, False, 0, "e4m3", 128, 16, "token"),
    ("bf16", 37, 4, 2, 128, 128, "half", 3, True, 0, "e4m3", 64, 16, "head"),
    ("f16", 250, 4, 1, 64, 64, "pair", 1, False, 0, "int8", 64, 32, "joined"),
    ("bf16", 9, 3, 3, 96, 64, "half", 2, True, 0, "int4", 32, 8, "token"),
    ("f32", 12, 2, 2, 256, 128, "half", 1, False, 0, "int8", 256, 16, "token"),
    ("f32", 12, 2, 1, 64, 64, "pair", 1, False, 0, "int4", 16, 16, "token"),
    ("f16", 7, 3, 1, 72, 36, "half", 1, False, 0, "int8", 24, 5, "token"),
    ("bf16", 7, 2, 1, 40, 10, "pair", 2, False, 1, "e4m3", 40, 5, "token"),
    ("bf16", 600, 2, 2, 128, 64, "half", 1, False, 0, "int4", 128, 64, "token"),
    ("f16", 5, 1, 1, 33, 32, "half", 1, False, 0, "int8", 3, 5, "token"),
    ("bf16", 6, 2, 2, 128, 96, "half", 1, False, 0, "e4m3", 8, 5, "token"),
    ("f16", 6, 2, 2, 72, 36, "half", 1, False, 0, "int4", 12, 5, "token"),
    ("bf16", 6, 3, 1, 64, 64, "pair", 1, False, 2, "int8", 2, 5, "head"),
    ("f16", 3, 2, 2, 128, 128, "pair", 1, False, 0, "int8", 32, 5, "token"),
    ("bf16", 3, 2, 2, 128, 128, "pair", 1, False, 0, "e4m3", 16, 5, "token"),
    ("bf16", 5003, 2, 1, 64, 64, "half", 1, True, 0, "int8", 32, 64, "head"),
    ("f16", 2601, 1, 1, 128, 128, "pair", 2, False, 0, "int4", 32, 64, "token"),
    ("bf16", 10003, 1, 1, 64, 32, "half", 1, False, 0, "e4m3", 16, 64, "token"),
]


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype,tokens,hq,hk,d,rot,pairs,axes,fused,offset,kind,group,page,layout", SERVED)
def test_serving_step_equals_its_parts(dtype, tokens, hq, hk, d, rot, pairs, axes, fused, offset, kind, group, page,
                                       layout, norm):
    c = Data(dtype, tokens, hq, hk, d, rot, axes, fused, offset, seed=3)
    pages = -(-tokens // page) + 1
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(4))[:tokens].cuda()
    if tokens > 3:
        slots[3] = -1
    how = dict(axis=c.axis, pairs=pairs)
    one, two = (make_cache(kind, pages, page, hk, d, group, layout) for _ in range(2))
    q1, k1, q2, k2, q3 = (c.place(torch.zeros_like(t), offset) for t in (c.q, c.k, c.q, c.k, c.q))
    if norm:
        nrm.nrm_qk_norm_rope_fwd(c.q, c.k, c.wq, c.wk, c.pos, c.inv, q1, k1, None, None, 1e-6, **how)
    else:
        nrm.nrm_rope_fwd(c.q, c.k, c.pos, c.inv, q1, k1, **how)
    nrm.nrm_kv_cache_write(k1, c.v, one, slots)
    nrm.nrm_qk_norm_rope_cache(c.q, c.k, c.v, c.wq, c.wk, c.pos, c.inv, q2, k2, two, slots, 1e-6, norm=norm, **how)
    nrm.nrm_sync_status()
    assert same(q1, q2) and same(k1, k2)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert same(getattr(one, n), getattr(two, n)), n
    # without the key itself, into a third cache
    three = make_cache(kind, pages, page, hk, d, group, layout)
    nrm.nrm_qk_norm_rope_cache(c.q, c.k, c.v, c.wq, c.wk, c.pos, c.inv, q3, None, three, slots, 1e-6, norm=norm, **how)
    assert same(q3, q1)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert same(getattr(one, n), getattr(three, n)), n


def test_a_served_sequence_in_chunks_equals_one_pass():
    # a prompt of 50 tokens, then single tokens, against all 60 at once: the same cache, the same context read back
    c = Data("bf16", 60, 4, 2, 128, 128, fused=True)
    table = torch.randperm(6, generator=torch.Generator().manual_seed(0)).cuda()
    t = torch.arange(60, device="cuda")
    slots = table[t // 16] * 16 + t % 16
    whole, parts = make_cache("int8", 6, 16, 2, 128, 64), make_cache("int8", 6, 16, 2, 128, 64)
    qo, qp = torch.empty(60, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(60, 4, 128, dtype=torch.bfloat16,
                                                                                     device="cuda")
    nrm.nrm_qk_norm_rope_cache(c.q, c.k, c.v, c.wq, c.wk, c.pos, c.inv, qo, None, whole, slots, 1e-6)
    for a, b in [(0, 50)] + [(i, i + 1) for i in range(50, 60)]:
        nrm.nrm_qk_norm_rope_cache(c.q[a:b], c.k[a:b], c.v[a:b], c.wq, c.wk, c.pos[:, a:b].contiguous(), c.inv, qp[a:b],
                                   None, parts, slots[a:b], 1e-6)
        back = [torch.empty(b, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        nrm.nrm_kv_cache_read(parts, slots[:b].contiguous(), *back)
    nrm.nrm_sync_status()
    assert same(qo, qp)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        assert same(getattr(whole, n), getattr(parts, n)), n
    # and the context is near what went in: half a code's step of its group, and bf16's rounding
    ko = torch.empty(60, 2, 128, dtype=torch.bfloat16, device="cuda")
    nrm.nrm_qk_norm_rope_fwd(c.q, c.k, c.wq, c.wk, c.pos, c.inv, qo, ko, None, None, 1e-6)
    for x, got in ((ko, back[0]), (c.v, back[1])):
        x, got = f64(x), f64(got)
        step = np.repeat(np.abs(x.reshape(60, 2, 2, 64)).max(-1) / 127, 64, -1).reshape(x.shape)
        assert (np.abs(x - got) <= 0.5001 * step + 2.0 ** -8 * np.abs(x) * 1.01).all()


def test_captured_step_follows_its_inputs():
    # a decode step in a CUDA graph, on a side stream: replays read the tensors' new contents
    s = torch.cuda.Stream()
    c = Data("bf16", 16, 8, 2, 128, 128)
    slots = torch.arange(16, device="cuda")
    cache = make_cache("e4m3", 2, 16, 2, 128, 128)
    qo = torch.empty_like(c.q)
    back = torch.empty_like(c.k), torch.empty_like(c.v)

    def step(cache, q_out, k_back, v_back):
        nrm.nrm_qk_norm_rope_cache(c.q, c.k, c.v, c.wq, c.wk, c.pos, c.inv, q_out, None, cache, slots, 1e-6)
        nrm.nrm_kv_cache_read(cache, slots, k_back, v_back)

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(cache, qo, *back)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step(cache, qo, *back)
    for i in range(3):
        c.q.normal_()
        c.k.normal_()
        c.pos.add_(1)
        slots.copy_(slots.flip(0) + (16 if i == 0 else 0))
        graph.replay()
        other = make_cache("e4m3", 2, 16, 2, 128, 128)
        q2, k2, v2 = torch.empty_like(qo), torch.empty_like(back[0]), torch.empty_like(back[1])
        step(other, q2, k2, v2)
        torch.cuda.synchronize()
        assert same(qo, q2) and same(back[0], k2) and same(back[1], v2)


def test_captured_backwards_with_workspaces_of_their_own():
    # two captured training steps replayed on two streams, and the same eagerly
    cases = [Data("bf16", 300, 4, 2, 128, 128, seed=i) for i in range(2)]
    outs = []
    streams = [torch.cuda.Stream() for _ in cases]
    graphs = []
    for c, s in zip(cases, streams):
        o = dict(qo=torch.empty_like(c.q), ko=torch.empty_like(c.k), dq=torch.empty_like(c.q), dk=torch.empty_like(c.k),
                 dwq=torch.empty_like(c.wq), dwk=torch.empty_like(c.wk), rq=torch.empty(300, 4, device="cuda"),
                 rk=torch.empty(300, 2, device="cuda"), ws=nrm.qk_norm_workspace(c.q))
        outs.append(o)
    torch.cuda.synchronize()

    def step(c, o):
        nrm.nrm_qk_norm_rope_fwd(c.q, c.k, c.wq, c.wk, c.pos, c.inv, o["qo"], o["ko"], o["rq"], o["rk"], 1e-6)
        nrm.nrm_qk_norm_rope_bwd(c.dqo, c.dko, c.q, c.k, c.wq, c.wk, o["rq"], o["rk"], c.pos, c.inv, o["dq"], o["dk"],
                                 o["dwq"], o["dwk"], o["ws"])

    want = []
    for c, o in zip(cases, outs):
        step(c, o)
        torch.cuda.synchronize()
        want.append({n: t.clone() for n, t in o.items() if n != "ws"})
    for c, o, s in zip(cases, outs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(c, o)
        graphs.append(g)
        for n, t in o.items():
            if n != "ws":
                t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for n in w:
            assert same(o[n], w[n]), n


def test_refusals_leave_the_context_usable():
    c = Data("bf16", 10, 2, 1, 64, 64)
    rq, rk = torch.empty(10, 2, device="cuda"), torch.empty(10, 1, device="cuda")
    qo, ko, dq, dk = (torch.empty_like(t) for t in (c.q, c.k, c.q, c.k))
    nrm.nrm_qk_norm_rope_fwd(c.q, c.k, c.wq, c.wk, c.pos, c.inv, qo, ko, rq, rk, 1e-6)
    ws = nrm.qk_norm_workspace(c.q)
    for bad in (None, ws[:-16], ws[4:]):
        with pytest.raises(nrm.NrmError) as e:
            nrm.nrm_qk_norm_rope_bwd(c.dqo, c.dko, c.q, c.k, c.wq, c.wk, rq, rk, c.pos, c.inv, dq, dk, torch.empty_like(c.wq),
                                     None, bad)
        assert e.value.status == nrm.NRM_ERR_WORKSPACE
    with pytest.raises(ValueError, match="current CUDA device"):
        nrm.nrm_qk_norm_rope_fwd(c.q, None, c.wq.cpu(), None, c.pos, c.inv, qo, None, None, None, 1e-6)
    with pytest.raises(ValueError, match="current CUDA device"):
        nrm.nrm_kv_cache_write(c.k, c.v, make_cache("int8", 2, 8, 1, 64, 64), torch.arange(10))
    nrm.nrm_sync_status()


# ---------------------------------------------------------------------------
# far offsets, other streams, first calls
# ---------------------------------------------------------------------------

def test_offsets_past_32_bits_in_a_long_cache():
    # 2^22 pages of 16 slots, 1 head of 128 in one byte each: 8 GiB of codes, the slots asked for beyond
    # 2^32 bytes and beyond 2^31
    pages = 1 << 22
    codes = torch.empty(pages, 16, 1, 128, dtype=torch.int8, device="cuda")
    scales = torch.empty(pages, 16, 1, 1, device="cuda")
    cache = nrm.kv_cache(codes, scales)
    slots = torch.tensor([0, (1 << 24) + 3, (1 << 25) + 5, pages * 16 - 1, 77], device="cuda")
    codes.view(-1, 128)[slots] = 0
    c = Data("bf16", 5, 1, 1, 128, 0)
    nrm.nrm_kv_cache_write(c.k, None, cache, slots)
    near = make_cache("int8", 1, 5, 1, 128, 128)
    nrm.nrm_kv_cache_write(c.k, None, near, torch.arange(5, device="cuda"))
    assert torch.equal(codes.view(-1, 128)[slots], near.k_codes.view(5, 128))
    assert torch.equal(scales.view(-1)[slots], near.k_scales.view(-1))
    a, b = torch.empty_like(c.k), torch.empty_like(c.k)
    nrm.nrm_kv_cache_read(cache, slots, a, None)
    nrm.nrm_kv_cache_read(near, torch.arange(5, device="cuda"), b, None)
    nrm.nrm_sync_status()
    assert same(a, b)


def test_offsets_past_32_bits_in_strided_views():
    # tokens 2^30 + 64 elements apart in one buffer of 6 GiB, forward and backward
    step = (1 << 30) + 64
    buf = torch.empty(2 * step + 3 * 256, dtype=torch.bfloat16, device="cuda")
    c = Data("bf16", 3, 2, 1, 128, 128)

    def far(t):
        v = buf.as_strided(t.shape, (step, 128, 1), 0)
        v.copy_(t)
        return v

    rq, r2 = torch.empty(3, 2, device="cuda"), torch.empty(3, 2, device="cuda")
    want, dq, dq2 = torch.empty_like(c.q), torch.empty_like(c.q), torch.empty_like(c.q)
    nrm.nrm_qk_norm_rope_fwd(c.q, None, c.wq, None, c.pos, c.inv, want, None, rq, None, 1e-6)
    nrm.nrm_qk_norm_rope_bwd(c.dqo, None, c.q, None, c.wq, None, rq, None, c.pos, c.inv, dq, None, None, None, None)
    v = far(c.q)
    nrm.nrm_qk_norm_rope_bwd(c.dqo, None, v, None, c.wq, None, rq, None, c.pos, c.inv, dq2, None, None, None, None)
    nrm.nrm_qk_norm_rope_fwd(v, None, c.wq, None, c.pos, c.inv, v, None, r2, None, 1e-6)
    nrm.nrm_sync_status()
    assert same(v, want) and same(rq, r2) and same(dq, dq2)


def test_calls_on_two_streams_at_once():
    cases = [Data("bf16", 3000, 8, 2, 128, 128, seed=i) for i in range(2)]
    caches = [make_cache("int8", 50, 64, 2, 128, 64, seed=i) for i in range(2)]
    slots = torch.randperm(3000, device="cuda")
    out = [torch.empty_like(c.q) for c in cases]
    back = [(torch.empty_like(c.k), torch.empty_like(c.v)) for c in cases]
    want = []
    for c, m, o, b in zip(cases, caches, out, back):
        nrm.nrm_qk_norm_rope_cache(c.q, c.k, c.v, c.wq, c.wk, c.pos, c.inv, o, None, m, slots, 1e-6)
        nrm.nrm_kv_cache_read(m, slots, *b)
        want.append([o.clone(), b[0].clone(), b[1].clone()])
        o.zero_(), b[0].zero_(), b[1].zero_()
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, c, m, o, b in zip(streams, cases, caches, out, back):
            nrm.nrm_qk_norm_rope_cache(c.q, c.k, c.v, c.wq, c.wk, c.pos, c.inv, o, None, m, slots, 1e-6, stream=s)
            with torch.cuda.stream(s):
                nrm.nrm_kv_cache_read(m, slots, *b)
    torch.cuda.synchronize()
    for o, b, w in zip(out, back, want):
        assert same(o, w[0]) and same(b[0], w[1]) and same(b[1], w[2])


FIRST_CALL = """
import torch, normalization_layernorm_rmsnorm_gb300 as nrm
q = torch.randn(4, 2, 64, device="cuda"); w = torch.ones(64, device="cuda"); o = torch.empty_like(q)
pos = torch.arange(4, device="cuda"); inv = torch.ones(32, device="cuda"); r = torch.empty(4, 2, device="cuda")
dq, dw = torch.empty_like(q), torch.empty_like(w); ws = nrm.qk_norm_workspace(q)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    nrm.nrm_qk_norm_rope_fwd(q, None, w, None, pos, inv, o, None, r, None, 1e-6)
    nrm.nrm_qk_norm_rope_bwd(o, None, q, None, w, None, r, None, pos, inv, dq, None, dw, None, ws)
g.replay(); torch.cuda.synchronize()
a, b = o.clone(), dw.clone(); o.zero_(); dw.zero_()
nrm.nrm_qk_norm_rope_fwd(q, None, w, None, pos, inv, o, None, r, None, 1e-6)
nrm.nrm_qk_norm_rope_bwd(o, None, q, None, w, None, r, None, pos, inv, dq, None, dw, None, ws)
nrm.nrm_sync_status()
assert torch.equal(a, o) and torch.equal(b, dw)
print("same")
"""


def test_a_first_call_may_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("norm,tokens,hq,hk,piece", [
    (True, 70_001, 12, 4, 4_999), (False, 70_001, 12, 4, 4_999), (True, 200_003, 1, 1, 30_011)])
def test_a_long_call_equals_its_pieces(norm, tokens, hq, hk, piece):
    # more tokens than the GPU holds at once several times over, against calls that it holds: a row's
    # result does not depend on the call that it is part of, so the bits are the same
    d, pages = 64, tokens // 16 + 7
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.randn(tokens, hq + 2 * hk, d, device="cuda", generator=g).bfloat16()
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    wq, wk = (torch.randn(d, device="cuda", generator=g).bfloat16() for _ in range(2))
    pos = torch.randint(0, 1 << 40, (tokens,), device="cuda", generator=g)
    inv = 0.5 ** torch.arange(d // 2, device="cuda").float()
    slots = torch.randperm(16 * pages, device="cuda", generator=g)[:tokens]

    def run(step):
        out = {"q": torch.zeros(tokens, hq, d, device="cuda", dtype=torch.bfloat16)}
        for n in ("k", "k_fused", "k_back", "v_back"):
            out[n] = torch.zeros(tokens, hk, d, device="cuda", dtype=torch.bfloat16)
        out["q_fused"] = torch.zeros_like(out["q"])
        codes = [torch.zeros(pages, 16, hk, d // 2, device="cuda", dtype=torch.uint8) for _ in range(4)]
        scales = [torch.zeros(pages, 16, hk, 2, device="cuda") for _ in range(4)]
        parts, fused = (nrm.kv_cache(codes[i], scales[i], codes[i + 1], scales[i + 1]) for i in (0, 2))
        for t in range(0, tokens, step):
            s = slice(t, t + step)
            if norm:
                nrm.nrm_qk_norm_rope_fwd(q[s], k[s], wq, wk, pos[s], inv, out["q"][s], out["k"][s], None, None, 1e-6)
            else:
                nrm.nrm_rope_fwd(q[s], k[s], pos[s], inv, out["q"][s], out["k"][s])
            nrm.nrm_kv_cache_write(out["k"][s], v[s], parts, slots[s])
            nrm.nrm_qk_norm_rope_cache(q[s], k[s], v[s], wq, wk, pos[s], inv, out["q_fused"][s], out["k_fused"][s], fused,
                                       slots[s], 1e-6, norm=norm)
            nrm.nrm_kv_cache_read(parts, slots[s], out["k_back"][s], out["v_back"][s])
        nrm.nrm_sync_status()
        out.update({f"codes{i}": c for i, c in enumerate(codes)})
        out.update({f"scales{i}": c for i, c in enumerate(scales)})
        return out

    whole, pieces = run(tokens), run(piece)
    for n, t in whole.items():
        assert torch.equal(t, pieces[n]), n
    assert torch.equal(whole["q"], whole["q_fused"]) and torch.equal(whole["k"], whole["k_fused"])
    for i in range(2):
        assert torch.equal(whole[f"codes{i}"], whole[f"codes{i + 2}"])
        assert torch.equal(whole[f"scales{i}"], whole[f"scales{i + 2}"])
    # and the last values: half a step of 4 bits off, then bf16's rounding (2^-8 of a value of at most 2 |x|)
    x = v[-7:].double().cpu().numpy()
    step = np.abs(x.reshape(7, hk, 2, 32)).max(-1, keepdims=True).repeat(32, -1).reshape(x.shape) / 7
    got = whole["v_back"][-7:].double().cpu().numpy()
    assert (np.abs(got - x) <= step * (0.5 + 1e-6) + np.abs(x) * 2.0 ** -7).all()


@pytest.mark.parametrize("captured", [False, True])
def test_calls_follow_other_streams_copies_and_kernels(captured):
    # each call is launched while its predecessor runs: what it waits for may be a copy, a fill, another
    # stream's kernel, or two of them at once, and what follows it on another stream waits for it
    tokens, heads, d = 3000, 4, 128
    g = torch.Generator(device="cuda").manual_seed(9)
    inv = 0.9 ** torch.arange(d // 2, device="cuda").float()
    pos = torch.arange(tokens, device="cuda")
    w = torch.randn(d, device="cuda", generator=g).bfloat16()
    src = [torch.empty(tokens, heads, d, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
    q, k, v, qo, ko, kb, vb, doubled = (torch.empty_like(src[0]) for _ in range(8))
    slots = torch.empty(tokens, dtype=torch.int64, device="cuda")
    order = torch.empty_like(slots)
    codes = [torch.zeros(tokens // 8, 8, heads, d, device="cuda", dtype=torch.int8) for _ in range(2)]
    scales = [torch.zeros(tokens // 8, 8, heads, 1, device="cuda") for _ in range(2)]
    cache = nrm.kv_cache(codes[0], scales[0], codes[1], scales[1])
    one, two = torch.cuda.Stream(), torch.cuda.Stream()

    def work():
        q.copy_(src[0])
        two.wait_stream(one)
        with torch.cuda.stream(two):
            k.copy_(src[1])
            k.mul_(2)
            v.copy_(src[2])
        q.mul_(2)
        one.wait_stream(two)
        nrm.nrm_qk_norm_rope_fwd(q, k, w, w, pos, inv, qo, ko, None, None, 1e-6)
        two.wait_stream(one)
        with torch.cuda.stream(two):
            torch.mul(ko, 2, out=doubled)
        slots.copy_(order)
        nrm.nrm_kv_cache_write(ko, v, cache, slots)
        kb.zero_()
        vb.zero_()
        nrm.nrm_kv_cache_read(cache, slots, kb, vb)
        one.wait_stream(two)

    torch.cuda.synchronize()
    if captured:
        for t in (*src, slots, order):
            t.zero_()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=one):
            work()
    for i in range(20):
        for t in src:
            t.copy_(torch.randn(t.shape, device="cuda", generator=g).bfloat16())
        order.copy_(torch.randperm(tokens, device="cuda", generator=g))
        torch.cuda.synchronize()
        if captured:
            graph.replay()
        else:
            with torch.cuda.stream(one):
                work()
        torch.cuda.synchronize()
        got = [t.clone() for t in (qo, ko, doubled, kb, vb)]
        q2, k2 = 2 * src[0], 2 * src[1]
        nrm.nrm_qk_norm_rope_fwd(q2, k2, w, w, pos, inv, qo, ko, None, None, 1e-6)
        torch.cuda.synchronize()
        nrm.nrm_kv_cache_write(ko, src[2], cache, order)
        torch.cuda.synchronize()
        nrm.nrm_kv_cache_read(cache, order, kb, vb)
        torch.cuda.synchronize()
        for a, b in zip(got, (qo, ko, 2 * ko, kb, vb)):
            assert torch.equal(a, b), i
    nrm.nrm_sync_status()
