"""The norms around a block with its gate and residual scale, forward and backward, against the
double-precision reference (oracle/served.py).

Tolerances, derived before the first run.  u = 2^-24 is half a step of float32; K = (cols/64 + 64) u
bounds a row's sum relative to the sum of its terms' sizes (at least 64 lanes share a row of more
than 64 columns, and a few levels join them).
  * r: K/2 from the sum of squares, 6 u for the root, the quotient and eps: R = K + 6 u.
  * y = x + alpha gate n: n off by R + 2 u, two products and the sum: (R + 6 u) |alpha gate n| + 2 u |y|.
  * h from the stored y: (R + 4 u) |h|.
  * dx = dy + r2 G - y c2, c2 = r2^3 s/cols with s off by K sum |G y|, G by u, and 6 products:
    8 u (|dy| + |r2 G| + |y c2|) + |y| r2^3/cols (K + 4 u) sum |G y|  =: E.
  * dn: |alpha gate| E + 4 u |dn|  =: F;  df = r1 g - f c1:  r1 |w| F + 8 u (r1 |g| + |f c1|) +
    |f| r1^3/cols (sum |w f| F + (K + 8 u) sum |g f|).
  * the columns' sums: each term's error, and (rows + 64) u of the terms' sizes.
Then half a step of the type.
"""
import numpy as np
import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
from oracle import served as ref
from test_heads import DT, TINY, U, f64, half_step, same, within

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    nrm.load()


class Block:
    def __init__(self, dtype, rows, cols, gates=0, alpha=1.0, post=True, pre=True, stream=True, weights=True, seed=0, offset=0,
                 loud=30.0):
        g = torch.Generator().manual_seed(seed + rows + 3 * cols)
        self.dtype, self.rows, self.cols, self.gates, self.alpha, self.post, self.pre = dtype, rows, cols, gates, alpha, post, pre
        self.offset, dt = offset, DT[dtype]

        def new(*shape, size=1.0, mean=0.0):
            return self.place((mean + size * torch.randn(*shape, generator=g)).to(dt))

        big = torch.ones(cols)
        big[cols // 3] = loud
        self.x, self.f = self.place((torch.randn(rows, cols, generator=g) * big).to(dt)), new(rows, cols, size=0.5)
        self.gate = new(gates, cols, size=0.7) if gates else None
        self.w_post = new(cols, size=0.2, mean=0.5) if post and weights else None
        self.w_pre = new(cols, size=0.2, mean=1.0) if pre and weights else None
        self.dh = new(rows, cols) if pre else None
        self.dy = new(rows, cols) if stream else None

    grads_at = None  # elements into their buffers; None: as all else

    def place(self, x, at=None):
        at = self.offset if at is None else at
        b = torch.empty(x.numel() + at, dtype=x.dtype, device="cuda")[at:].view(x.shape)
        b.copy_(x)
        return b

    def like(self, x, at=None):
        return None if x is None else self.place(torch.full(x.shape, 7.0, dtype=x.dtype), at)

    def fwd(self, y=None, h=None, stats=True, stream=None):
        y = self.like(self.x) if y is None else y
        h = (self.like(self.x) if h is None else h) if self.pre else None
        r1 = torch.full((self.rows,), 7.0, device="cuda") if stats and self.post else None
        r2 = torch.full((self.rows,), 7.0, device="cuda") if stats and self.pre else None
        nrm.nrm_block_norm_fwd(self.x, self.f, self.gate, self.w_post, self.w_pre, y, h, r1, r2, self.alpha, EPS,
                               post=self.post, stream=stream)
        return y, h, r1, r2

    def bwd(self, y, r1, r2, grads=True, ws=None, stream=None):
        dx, df = self.like(self.x), self.like(self.x)
        dgate, dw1, dw2 = (self.like(t, self.grads_at) if grads else None for t in (self.gate, self.w_post, self.w_pre))
        if ws is None and grads:
            ws = nrm.block_norm_workspace(self.x, self.gate)
            ws.fill_(0xff)
        nrm.nrm_block_norm_bwd(self.dh, self.dy, self.f, y, self.gate, self.w_post, self.w_pre, r1, r2, dx, df, dgate, dw1, dw2,
                               ws, self.alpha, post=self.post, stream=stream)
        return dx, df, dgate, dw1, dw2

    def check(self):
        o = {n: None if getattr(self, n) is None else f64(getattr(self, n)) for n in ("x", "f", "gate", "w_post", "w_pre", "dh", "dy")}
        K = (self.cols / 64 + 64) * U
        R = K + 6 * U
        y, h, r1, r2 = self.fwd()
        want_y, want_r1 = ref.block_fwd(o["x"], o["f"], o["gate"], o["w_post"], self.alpha, EPS, self.post)
        part = np.abs(want_y - o["x"])
        within(y, want_y, (R + 6 * U) * part + 2 * U * (np.abs(o["x"]) + part), self.dtype, "y")
        if self.post:
            assert (np.abs(f64(r1) - want_r1) <= R * want_r1).all()
        yy = f64(y)
        if self.pre:
            want_h, want_r2 = ref.block_pre(yy, o["w_pre"], EPS)
            within(h, want_h, (R + 4 * U) * np.abs(want_h), self.dtype, "h")
            assert (np.abs(f64(r2) - want_r2) <= R * want_r2).all()
        if self.dh is None and self.dy is None:
            return
        a1 = f64(r1) if self.post else None
        a2 = f64(r2) if self.pre else None
        dx, df, dgate, dw1, dw2 = self.bwd(y, r1, r2)
        w = ref.block_bwd(o["dh"], o["dy"], o["f"], yy, o["gate"], o["w_post"], o["w_pre"], a1, a2, self.alpha, self.post)
        n = self.cols
        E = 8 * U * (np.abs(o["dy"]) if o["dy"] is not None else 0.0) + np.zeros_like(o["f"])
        if self.pre:
            r = a2[:, None]
            G = np.abs(o["dh"] * (1.0 if o["w_pre"] is None else o["w_pre"]))
            terms = (G * np.abs(yy)).sum(-1, keepdims=True)
            c2 = r ** 3 * terms / n
            E = E + 8 * U * (r * G + np.abs(yy) * c2) + np.abs(yy) * r ** 3 / n * (K + 4 * U) * terms
        within(dx, w[0], E, self.dtype, "dx")
        ag = np.abs(self.alpha * ref._spread(o["gate"], self.rows))
        dn = ag * np.abs(w[0])
        F = ag * E + 4 * U * dn
        lim = F
        if self.post:
            r = a1[:, None]
            wf = np.abs(1.0 if o["w_post"] is None else o["w_post"]) * np.ones(n)
            g, fa = dn * wf, np.abs(o["f"])
            terms = (g * fa).sum(-1, keepdims=True)
            lim = r * wf * F + 8 * U * (r * g + fa * r ** 3 / n * terms) + fa * r ** 3 / n * (
                (wf * fa * F).sum(-1, keepdims=True) + (K + 8 * U) * terms)
        within(df, w[1], lim, self.dtype, "df")
        many = (self.rows + 64) * U
        unit = np.abs(o["f"]) * (a1[:, None] if self.post else 1.0)
        if self.gate is not None:
            n1 = unit * np.abs(1.0 if not self.post or o["w_post"] is None else o["w_post"])
            err = np.abs(self.alpha) * n1 * (E + (many + 8 * U) * np.abs(w[0]))
            within(dgate, w[2], err.reshape(self.gates, -1, n).sum(1), self.dtype, "dgate")
        if dw1 is not None:
            within(dw1, w[3], (unit * (F + (many + 8 * U) * dn)).sum(0), self.dtype, "dw_post")
        if dw2 is not None:
            within(dw2, w[4], ((many + 8 * U) * np.abs(o["dh"] * yy) * a2[:, None]).sum(0), self.dtype, "dw_pre")


SHAPES = [
    # dtype, rows, cols, gates
    ("bf16", 1, 4096, 0), ("bf16", 1, 4096, 1), ("bf16", 300, 4096, 1), ("f16", 394, 768, 2), ("f16", 7, 768, 7), ("f32", 33, 1000, 1),
    ("f32", 640, 256, 320), ("f32", 640, 256, 640), ("bf16", 2000, 64, 5), ("f16", 45, 8192, 3), ("bf16", 24, 12000, 4),
    ("f32", 9, 8192, 1), ("f16", 40, 16384, 1), ("bf16", 4, 40000, 2), ("bf16", 33, 777, 3), ("f16", 12, 1, 4), ("f32", 5, 3, 0),
    ("f32", 100, 2, 50), ("bf16", 100, 8, 1), ("f16", 1000, 96, 1000), ("f32", 50, 4100, 1), ("bf16", 610, 2048, 305),
    ("bf16", 50, 2056, 1), ("f16", 1, 24, 1), ("f16", 50, 520, 10),
]


@pytest.mark.parametrize("dtype,rows,cols,gates", SHAPES)
def test_against_the_reference(dtype, rows, cols, gates):
    Block(dtype, rows, cols, gates, alpha=0.5).check()


@pytest.mark.parametrize("dtype,cols", [("bf16", 1024), ("f32", 600), ("f16", 333), ("bf16", 9000)])
@pytest.mark.parametrize("gates", [0, 1, 6])
@pytest.mark.parametrize("post,pre,stream", [(True, True, False), (True, False, True), (False, True, True), (False, False, True),
                                             (False, True, False)])
def test_parts_left_out(dtype, cols, gates, post, pre, stream):
    Block(dtype, 66, cols, gates, alpha=-1.5, post=post, pre=pre, stream=stream).check()


@pytest.mark.parametrize("cols", [1024, 333, 9000])
def test_without_weights(cols):
    Block("f32", 20, cols, 1, weights=False).check()
    b = Block("bf16", 20, cols, 2)
    y, h, r1, r2 = b.fwd()
    y2, h2, _, _ = b.fwd(stats=False)
    assert same(y, y2) and same(h, h2)
    all_ = b.bwd(y, r1, r2)
    assert all(same(p, q) for p, q in zip(b.bwd(y, r1, r2, grads=False)[:2], all_[:2]))
    # one gradient alone is the same bits
    ws = nrm.block_norm_workspace(b.x, b.gate)
    for i, name in enumerate(("dgate", "dw_post", "dw_pre")):
        one = {n: b.like(t) if n == name else None for n, t in (("dgate", b.gate), ("dw_post", b.w_post), ("dw_pre", b.w_pre))}
        nrm.nrm_block_norm_bwd(b.dh, b.dy, b.f, y, b.gate, b.w_post, b.w_pre, r1, r2, b.like(b.x), b.like(b.x), one["dgate"],
                               one["dw_post"], one["dw_pre"], ws, b.alpha)
        assert same(one[name], all_[2 + i])


@pytest.mark.parametrize("offset", [1, 4])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_unaligned(dtype, offset):
    Block(dtype, 30, 512, 3, offset=offset).check()


@pytest.mark.parametrize("cols", [4096, 777, 20000])
def test_in_place(cols):
    b = Block("bf16", 37, cols, 1)
    y, h, r1, r2 = b.fwd()
    x, f = b.x.clone(), b.f.clone()
    y2, h2, _, _ = b.fwd(y=b.x, h=b.f)
    assert y2 is b.x and same(y, b.x) and same(h, b.f)
    b.x, b.f = x, f
    b.fwd(y=b.x)
    assert same(y, b.x)


@pytest.mark.parametrize("cols", [1024, 100])
def test_the_unfused_calls_agree(cols):
    # y is what the next norm takes, as it is stored; without the norm after the block and alpha = 1, gate 1: the plain sum
    b = Block("bf16", 50, cols, 0, post=False)
    y, h, _, r2 = b.fwd()
    assert same(y, b.x + b.f)
    want, r = torch.empty_like(y), torch.empty_like(r2)
    nrm.nrm_rmsnorm_fwd(y, b.w_pre, want, r, EPS)
    # the sums may be added in another order
    assert torch.allclose(h.float(), want.float(), rtol=2 ** -7, atol=0) and torch.allclose(r, r2, rtol=1e-6)


@pytest.mark.parametrize("cols", [1024, 333, 9000])
def test_rows_of_special_values(cols):
    b = Block("f32", 12, cols, 1)
    b.f[0] = 0
    b.x[1] = 0
    b.x[2] = b.f[2] = 0
    b.f[3, 5] = float("nan")
    b.x[4, 5] = float("inf")
    y, h, r1, r2 = b.fwd()
    assert (r1[0] == r1[2]) and abs(float(r1[0]) - EPS ** -0.5) < 1e-3 and not h[2].any() and not y[2].any()
    assert y[3].isnan().all() and h[3].isnan().all() and y[4, 5].isinf() and h[4, 5].isnan()
    rest = [0, 1, 2, 5, 6, 7, 8, 9, 10, 11]
    assert y[rest].isfinite().all() and h[rest].isfinite().all()
    dx, df, *_ = b.bwd(y, r1, r2)
    assert dx[rest].isfinite().all() and df[rest].isfinite().all() and dx[3].isnan().all()


def test_no_rows():
    b = Block("bf16", 0, 64, 0)
    y, h, r1, r2 = b.fwd()
    dx, df, _, dw1, dw2 = b.bwd(y, r1, r2)
    assert not dw1.any() and not dw2.any()
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    gate, dgate = torch.ones(3, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(3, 64, dtype=torch.bfloat16, device="cuda")
    nrm.nrm_block_norm_bwd(e, e, e, e, gate, None, None, r1, r2, e, e, dgate, None, None, None, 1.0)
    assert not dgate.any()


def test_gradients_against_differences():
    # of the call itself, in float32: loss = sum(dh h + dy y), central differences of step 2^-6
    b = Block("f32", 6, 40, 2, alpha=0.7, loud=1.0)
    y, _, r1, r2 = b.fwd()
    got = b.bwd(y, r1, r2)

    def loss():
        yy, hh, _, _ = b.fwd()
        return float((b.dh.double() * hh.double() + b.dy.double() * yy.double()).sum())

    step = 2.0 ** -6
    for t, grad in ((b.x, got[0]), (b.f, got[1]), (b.gate, got[2]), (b.w_post, got[3]), (b.w_pre, got[4])):
        flat, g = t.view(-1), grad.view(-1)
        for i in range(0, flat.numel(), max(1, flat.numel() // 17)):
            keep = float(flat[i])
            flat[i] = keep + step
            up = loss()
            flat[i] = keep - step
            down = loss()
            flat[i] = keep
            # truncation: step^2 / 6 of a third derivative of a few units; rounding: 240 outputs of a few u, over 2 steps
            assert abs((up - down) / (2 * step) - float(g[i])) < 0.01 + 0.01 * abs(float(g[i])), (i, up, down, float(g[i]))


@pytest.mark.parametrize("rows,cols,gates", [(1030, 4096, 1), (985, 768, 5), (1000, 1536, 500), (700, 512, 0), (1300, 96, 13), (3000, 4096, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows(dtype, rows, cols, gates):
    # every slot of the ring used many times over, chunks that begin inside a gate's rows, rows that do not fill a slot
    Block(dtype, rows, cols, gates, alpha=0.5).check()


@pytest.mark.parametrize("gates", [2, 64, 320, 640])
def test_gates_of_few_rows(gates):
    Block("bf16", 640, 256, gates).check()
    Block("f32", 640, 256, gates, pre=False).check()
    Block("f16", 640, 256, gates, post=False, stream=False).check()


def test_captured_with_a_shared_workspace():
    blocks = [Block("bf16", 700, 512, g, seed=g) for g in (1, 7)]
    ws = torch.empty(max(nrm.block_norm_workspace(b.x, b.gate).numel() for b in blocks), dtype=torch.uint8, device="cuda")
    want, graphs, outs = [], [], []
    for b in blocks:
        y, h, r1, r2 = b.fwd()
        want.append((y, h, *b.bwd(y, r1, r2)))
    torch.cuda.synchronize()
    for b in blocks:
        dx, df = torch.empty_like(b.x), torch.empty_like(b.x)
        grads = [torch.empty_like(t) for t in (b.gate, b.w_post, b.w_pre)]
        y, h, r1, r2 = torch.empty_like(b.x), torch.empty_like(b.x), torch.empty(700, device="cuda"), torch.empty(700, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nrm.nrm_block_norm_fwd(b.x, b.f, b.gate, b.w_post, b.w_pre, y, h, r1, r2, b.alpha, EPS)
            nrm.nrm_block_norm_bwd(b.dh, b.dy, b.f, y, b.gate, b.w_post, b.w_pre, r1, r2, dx, df, *grads, ws, b.alpha)
        graphs.append(graph)
        outs.append((y, h, dx, df, *grads))
    for _ in range(10):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for got, exp in zip(outs, want):
        assert all(same(p, q) for p, q in zip(got, exp))


def test_the_same_bits_again_on_another_stream():
    b = Block("bf16", 1500, 1024, 1)
    y, h, r1, r2 = b.fwd()
    first = b.bwd(y, r1, r2)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y2, h2, s1, s2 = b.fwd(stream=st)
    again = b.bwd(y2, s1, s2, stream=st)
    torch.cuda.synchronize()
    assert same(y, y2) and same(h, h2) and all(same(p, q) for p, q in zip(first, again))


@pytest.mark.parametrize("seed", range(40))
def test_random_shapes(seed):
    rng = np.random.default_rng(seed)
    step = int(rng.choice([1, 2, 8, 64]))
    cols = max(step, int(2 ** rng.uniform(0, 14)) // step * step)
    gates = int(rng.choice([0, 1, rng.integers(1, 40)]))
    per = int(2 ** rng.uniform(0, 7))
    rows = max(1, gates) * per if gates > 1 else int(2 ** rng.uniform(0, 10))
    rows = min(rows, max(1, (1 << 21) // cols) // max(1, gates) * max(1, gates)) or max(1, gates)
    Block(str(rng.choice(["bf16", "f16", "f32"])), rows, cols, gates, alpha=float(rng.choice([1.0, 0.5, -2.0])), post=bool(rng.random() < 0.8),
          pre=bool(rng.random() < 0.9), seed=seed, weights=bool(rng.random() < 0.9)).check()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,gates", [(30, 3), (30, 30), (400, 1), (400, 2)])
def test_unaligned_gradients_alone(dtype, rows, gates):
    # all else is whole vectors
    c = Block(dtype, rows, 512, gates)
    c.grads_at = 1
    c.check()
    nrm.nrm_sync_status()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols,gates", [
    (61, 67, 0), (61, 67, 1), (60, 67, 60), (60, 250, 4), (40, 513, 2), (40, 1001, 40), (45, 1023, 3), (30, 2049, 1), (18, 4095, 2),
    (18, 4097, 18), (10, 6001, 1), (10, 8191, 5), (6, 8193, 1), (300, 1001, 1), (3000, 131, 6), (390, 80, 130), (1, 1, 0), (1, 5, 1), (3, 2, 3),
])
def test_odd_rows_of_every_kernel(dtype, rows, cols, gates):
    # rows that begin anywhere within 16 bytes, and tensors that end there
    Block(dtype, rows, cols, gates).check()
    nrm.nrm_sync_status()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_odd_rows_leave_what_lies_around_them(dtype):
    # the copies are rounded outwards: neither inputs nor what lies before and behind the outputs may change, and
    # what lies around the inputs may be anything
    rows, cols = 29, 333
    c = Block(dtype, rows, cols, 1)
    y, _, r1, r2 = c.fwd()
    want = c.bwd(y, r1, r2)

    def inside(x, around):
        b = torch.full((x.numel() + 32,), around, dtype=x.dtype, device="cuda")
        b[16:16 + x.numel()].view(x.shape).copy_(x)
        return b, b[16:16 + x.numel()].view(x.shape)

    for name in ("x", "f", "dh", "dy"):
        setattr(c, name, inside(getattr(c, name), float("nan"))[1])
    y = inside(y, float("inf"))[1]
    outs = [inside(t, 7.0) for t in want]
    ws = nrm.block_norm_workspace(c.x, c.gate)
    nrm.nrm_block_norm_bwd(c.dh, c.dy, c.f, y, c.gate, c.w_post, c.w_pre, r1, r2, *[v for _, v in outs], ws, c.alpha)
    nrm.nrm_sync_status()
    for (b, v), w in zip(outs, want):
        assert same(v.contiguous(), w) and (b[:16] == 7).all() and (b[16 + w.numel():] == 7).all()
