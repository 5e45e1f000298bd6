"""Calls on heads that keep every warp (or CTA) busy for many steps: places in the rings of copies
are used again and again, and a lane adds many rows to its sums.

The backward's dx belongs to its row alone, so a long call gives the bits of its pieces.  Its dw is
  * exact where every term is a small whole number (rows of -2..2, gradients of -2..2, r = 1/2, no
    turn, sums below 2^22): equal, so that no row may be lost or added twice;
  * else off by 24 u a term (the products and the turn), and by the chains that add the terms: a lane's
    rows, then 5 levels of the warp, 8 warps and the partial rows with their rounding carried:
    (24 + rows of a lane + 40) u sum G'|x| r, and half a step of the type it is stored in.
A lane's rows are at most what one CTA of eight warps an SM would leave it."""
import numpy as np
import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    nrm.load()


LONG = [
    # dtype, tokens, hq, hk, d, rot, pairs, axes, offset (elements), piece
    ("bf16", 16411, 32, 8, 128, 128, "half", 1, 0, 4099),  # one token a warp, the keys' heads in one step
    ("f16", 30011, 16, 16, 64, 64, "pair", 2, 0, 7001),
    ("f32", 12007, 12, 4, 80, 40, "half", 3, 0, 2999),     # 16-byte vectors of float32
    ("bf16", 60013, 8, 2, 64, 32, "half", 1, 0, 9001),     # several tokens a warp for the keys only
    ("f16", 120011, 1, 1, 64, 64, "pair", 1, 0, 30011),    # ... and for both
    ("f32", 90007, 2, 1, 32, 32, "half", 1, 0, 20011),
    ("bf16", 30011, 4, 4, 72, 36, "half", 1, 0, 5003),     # 4-byte vectors
    ("f16", 20011, 6, 2, 72, 72, "half", 1, 0, 5003),      # 8-byte vectors
    ("bf16", 9001, 7, 3, 33, 16, "half", 2, 0, 2003),      # element by element: 1, 2 and 4 slots a lane
    ("f16", 9001, 5, 2, 96, 50, "pair", 1, 1, 2003),
    ("f32", 9001, 3, 3, 255, 254, "half", 1, 0, 2003),
]
NAMES = "dtype,tokens,hq,hk,d,rot,pairs,axes,offset,piece"


class Call:
    def __init__(self, dtype, tokens, hq, hk, d, rot, pairs, axes, offset, whole):
        g = torch.Generator(device="cuda").manual_seed(tokens)
        self.dt, self.tokens, self.heads, self.d, self.rot = DT[dtype], tokens, (hq, hk), d, rot

        def rows(heads, fused=False):
            if whole:
                x = torch.randint(-2, 3, (tokens, heads, d), device="cuda", generator=g, dtype=torch.int32).to(self.dt)
            else:
                x = torch.randn(tokens, heads, d, device="cuda", generator=g).to(self.dt)
            if offset:
                b = torch.empty(x.numel() + offset, device="cuda", dtype=self.dt)[offset:].view(x.shape)
                return b.copy_(x)
            return x

        qkv = rows(hq + 2 * hk)  # a fused projection
        self.x = [qkv[:, :hq], qkv[:, hq:hq + hk]]
        self.dy = [rows(hq), rows(hk)]
        self.w = [torch.ones(d, device="cuda", dtype=self.dt) if whole else
                  (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(self.dt) for _ in range(2)]
        self.r = [torch.full((tokens, h), 0.5, device="cuda") if whole else
                  ((t.double() ** 2).mean(-1) + 1e-6).rsqrt().float().contiguous() for h, t in zip((hq, hk), self.x)]
        self.pos = torch.randint(0, 9000, (axes, tokens), device="cuda", generator=g)
        if whole:
            self.pos.zero_()
        self.inv = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))).float().cuda()
        self.axis_of = torch.tensor([p % axes for p in range(rot // 2)], device="cuda")
        self.how = dict(axis=bytes(self.axis_of.tolist()) if axes > 1 else None, pairs=pairs)
        self.dx = [torch.zeros(tokens, h, d, device="cuda", dtype=self.dt) for h in (hq, hk)]
        self.dw = [torch.zeros(d, device="cuda", dtype=self.dt) for _ in range(2)]
        self.ws = nrm.qk_norm_workspace(self.x[0])

    def bwd(self, s=slice(None)):
        nrm.nrm_qk_norm_rope_bwd(self.dy[0][s], self.dy[1][s], self.x[0][s], self.x[1][s], *self.w, self.r[0][s], self.r[1][s],
                                 self.pos[:, s].contiguous(), self.inv, self.dx[0][s], self.dx[1][s], *self.dw, self.ws,
                                 **self.how)
        nrm.nrm_sync_status()

    def turned_back(self, which):
        """(R^T dy, and |a| + |b| of each element's pair) in float64"""
        dy = self.dy[which].double()
        a = (self.pos[self.axis_of].t().double() * self.inv.double())[:, None]
        n = self.rot // 2
        i, j = (slice(0, n), slice(n, 2 * n)) if self.how["pairs"] == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
        back, size = dy.clone(), dy.abs()
        back[..., i] = dy[..., i] * a.cos() + dy[..., j] * a.sin()
        back[..., j] = dy[..., j] * a.cos() - dy[..., i] * a.sin()
        both = size[..., i] + size[..., j]
        size[..., i], size[..., j] = both, both
        return back, size


@pytest.mark.parametrize(NAMES, LONG)
def test_a_long_backward(dtype, tokens, hq, hk, d, rot, pairs, axes, offset, piece):
    c = Call(dtype, tokens, hq, hk, d, rot, pairs, axes, offset, False)
    c.bwd()
    dx, dw = [t.clone() for t in c.dx], [t.clone() for t in c.dw]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for i, tag in enumerate("qk"):
        back, size = c.turned_back(i)
        x, r = c.x[i].double(), c.r[i].double()[..., None]
        want = (back * x * r).sum((0, 1))
        # one row of a warp at least, and one eighth of the CTAs at least for either tensor
        lane = tokens * c.heads[i] * 8 / (8 * sms) + 1
        lim = (24 + lane + 40) * U * (size * x.abs() * r).sum((0, 1))
        lim += torch.finfo(c.dt).eps / 2 * (want.abs() + lim)
        assert ((dw[i].double() - want).abs() <= lim).all(), f"dw{tag}"
        # dx = r g - x r^3 s/d, to 24 u r G of the first term and 80 u |x| r^3 sum G|x| / d of the second
        g, gs = back * c.w[i].double(), size * c.w[i].double().abs()
        want = r * g - x * r ** 3 * (g * x).mean(-1, keepdim=True)
        lim = U * (24 * r * gs + 80 * x.abs() * r ** 3 * (gs * x.abs()).mean(-1, keepdim=True))
        lim += torch.finfo(c.dt).eps / 2 * (want.abs() + lim) + torch.finfo(c.dt).smallest_normal * torch.finfo(c.dt).eps / 2
        assert ((dx[i].double() - want).abs() <= lim).all(), f"d{tag}"
    for t in c.dx:
        t.zero_()
    for t in range(0, tokens, piece):
        c.bwd(slice(t, t + piece))
    for i, tag in enumerate("qk"):
        assert torch.equal(dx[i].view(torch.uint8), c.dx[i].view(torch.uint8)), f"d{tag} differs from its pieces"


@pytest.mark.parametrize(NAMES, LONG)
def test_a_long_backward_adds_every_row_once(dtype, tokens, hq, hk, d, rot, pairs, axes, offset, piece):
    c = Call(dtype, tokens, hq, hk, d, rot, pairs, axes, offset, True)
    c.bwd()
    for i in range(2):
        exact = (c.dy[i].double() * c.x[i].double()).sum((0, 1)) * 0.5
        assert exact.abs().max() < 2 ** 22
        assert torch.equal(c.dw[i], exact.to(c.dt)), "qk"[i]


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype,tokens,hq,hk,d,rot,offset,kind,group", [
    ("bf16", 20011, 7, 3, 33, 16, 0, "int8", 11),
    ("f16", 20011, 5, 2, 96, 50, 1, "e4m3", 96),
    ("f32", 20011, 3, 3, 256, 254, 0, "int4", 64),
    ("bf16", 60013, 6, 2, 72, 36, 0, "int8", 36),
    ("f32", 40009, 4, 2, 80, 80, 0, "e4m3", 40),
])
def test_a_long_forward_and_cache_equal_their_pieces(dtype, tokens, hq, hk, d, rot, offset, kind, group, norm):
    # layouts that take narrower accesses or single elements
    g = torch.Generator(device="cuda").manual_seed(d)
    dt, page = DT[dtype], 16
    pages = tokens // page + 3
    buf = torch.empty(tokens * (hq + 2 * hk) * d + offset, device="cuda", dtype=dt)
    qkv = buf[offset:].view(tokens, hq + 2 * hk, d)
    qkv.copy_(torch.randn(qkv.shape, device="cuda", generator=g))
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    w = torch.randn(d, device="cuda", generator=g).to(dt)
    pos = torch.randint(0, 1 << 33, (tokens,), device="cuda", generator=g)
    inv = 0.7 ** torch.arange(rot // 2, device="cuda").float()
    slots = torch.randperm(page * pages, device="cuda", generator=g)[:tokens]
    code = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8, "int4": torch.uint8}[kind]
    width = d // 2 if kind == "int4" else d

    def run(step):
        out = {n: torch.zeros(tokens, h, d, device="cuda", dtype=dt)
               for n, h in (("q", hq), ("k", hk), ("qf", hq), ("kf", hk), ("kb", hk), ("vb", hk))}
        codes = [torch.zeros(pages, page, hk, width, device="cuda", dtype=torch.uint8).view(code) for _ in range(4)]
        scales = [torch.zeros(pages, page, hk, d // group, device="cuda") for _ in range(4)]
        parts, fused = (nrm.kv_cache(codes[i], scales[i], codes[i + 1], scales[i + 1]) for i in (0, 2))
        for t in range(0, tokens, step):
            s = slice(t, t + step)
            if norm:
                nrm.nrm_qk_norm_rope_fwd(q[s], k[s], w, w, pos[s], inv, out["q"][s], out["k"][s], None, None, 1e-6)
            else:
                nrm.nrm_rope_fwd(q[s], k[s], pos[s], inv, out["q"][s], out["k"][s])
            nrm.nrm_kv_cache_write(out["k"][s], v[s], parts, slots[s])
            nrm.nrm_qk_norm_rope_cache(q[s], k[s], v[s], w, w, pos[s], inv, out["qf"][s], out["kf"][s], fused, slots[s], 1e-6,
                                       norm=norm)
            nrm.nrm_kv_cache_read(parts, slots[s], out["kb"][s], out["vb"][s])
        nrm.nrm_sync_status()
        out |= {f"codes{i}": t.view(torch.uint8) for i, t in enumerate(codes)}
        return out | {f"scales{i}": t for i, t in enumerate(scales)}

    whole, pieces = run(tokens), run(2003)
    for n, t in whole.items():
        assert torch.equal(t.view(torch.uint8), pieces[n].view(torch.uint8)), n
