"""Attention over the paged cache through libnorm's public call, against the double-precision
reference (oracle/served.py).

Tolerances, derived before the first run.  u = 2^-24 is half a step of float32.
  * A logit is a float32 sum of d exact products (of factors with 22 bits for float32 queries:
    2^-21 of each) in any order, each addition off by at most a step, 2u (the tensor cores cut
    off), then three products: |dl| <= D = (2 (d + 16) u + 2^-21) S + 8 u |l|, S = sum |q k| scale;
    in base 2 and back it is held in float32: 2 u (|l| + |lse|) more, counted in the 8 and below.
  * p = 2^(l - m) and its sum: the exponent's error, 2 D, the function's 2^-21, and n additions:
    a relative 2 D + 2^-21 + 2 (n + 64) u each, twice for the quotient.
  * out: n more products and additions, and for bfloat16 the weights are rounded to 11 bits:
    2^-11 at most; what lies below 2^-38 of the largest term is lost.
  * Then half a step of the output's type.
"""
import numpy as np
import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
from oracle import served as ref
from test_heads import CODES, DT, TINY, U, f64, half_step, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    nrm.load()


class Case:
    """A cache with sequences on pages in no order; the slots that no position has are poison."""

    def __init__(self, dtype, lengths, hq, hk, d, kind="e4m3", group=None, page=16, width=None, seed=0, order="pshd",
                 offset=0, poison=float("nan"), loud=1.0):
        g = torch.Generator().manual_seed(seed + 7 * d + len(lengths))
        self.dtype, self.kind, self.page, self.hq, self.hk, self.d = dtype, kind, page, hq, hk, d
        group = group or d
        self.lengths = torch.tensor(lengths, dtype=torch.int64)
        seqs = len(lengths)
        width = width or max(1, -(-max([0, *lengths]) // page))
        pages = seqs * width + 2
        self.table = torch.randperm(pages, generator=g)[:seqs * width].view(seqs, width)
        used = torch.zeros(pages, page, dtype=torch.bool)
        for s, n in enumerate(lengths):
            j = torch.arange(max(0, min(n, width * page)))
            used[self.table[s, j // page], j % page] = True
        self.codes, self.scales = [], []
        for t in range(2):
            scales = torch.rand(pages, page, hk, d // group, generator=g) / {"e4m3": 200, "int8": 60, "int4": 4}[kind]
            if kind == "e4m3":
                codes = (torch.randn(pages, page, hk, d, generator=g) * 120).clamp(-448, 448).to(torch.float8_e4m3fn)
                codes.view(torch.uint8)[~used] = 0x7f  # a NaN
            elif kind == "int8":
                codes = torch.randint(-127, 128, (pages, page, hk, d), generator=g).to(torch.int8)
            else:
                low, high = (torch.randint(-7, 8, (pages, page, hk, d // 2), generator=g) & 15 for _ in range(2))
                codes = (low | high << 4).to(torch.uint8)
            scales[~used] = poison
            self.codes.append(self.lay(codes, order, offset))
            self.scales.append(self.lay(scales, order, 0))
        self.q = (torch.randn(seqs, hq, d, generator=g) * loud).to(DT[dtype])
        self.cache = nrm.kv_cache(self.codes[0], self.scales[0], self.codes[1], self.scales[1])

    @staticmethod
    def lay(t, order, offset):
        """t [pages, page, heads, d] on the GPU, in memory as `order` says, `offset` bytes into its buffer."""
        perm = ["pshd".index(c) for c in order]
        x = t.permute(perm).contiguous()
        raw = torch.zeros(x.numel() * x.element_size() + 64, dtype=torch.uint8, device="cuda")
        raw = raw[offset:offset + x.numel() * x.element_size()]
        raw.copy_(x.view(torch.uint8).flatten())
        return raw.view(x.dtype).view(x.shape).permute([perm.index(i) for i in range(4)])

    def values(self, t):
        codes = self.codes[t].cpu()
        codes = codes.float().numpy() if self.kind != "int4" else codes.numpy()
        return ref.stored(codes, self.scales[t].cpu().numpy(), self.kind)

    def run(self, window=0, weights=None, lse=False, scale=None, q=None, out=None, stream=None):
        q = self.q.cuda() if q is None else q
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda") if out is None else out
        got_lse = torch.empty(q.shape[:2], device="cuda") if lse else None
        ws = nrm.kv_attention_workspace(q, self.cache, self.table, weights=weights is not None)
        ws.fill_(0xff)
        nrm.nrm_kv_cache_attention(q, self.cache, self.table.cuda(), self.lengths.cuda(), out,
                                   self.d ** -0.5 if scale is None else scale, ws, window=window, lse=got_lse,
                                   weights=weights, stream=stream)
        return out, got_lse

    def check(self, window=0, weights=False, scale=None, **kw):
        scale = self.d ** -0.5 if scale is None else scale
        cap = self.table.shape[1] * self.page
        before = torch.rand(len(self.lengths), self.hk, cap, generator=torch.Generator().manual_seed(1)) if weights else None
        w = before.cuda() if weights else None
        out, lse = self.run(window, w, True, scale, **kw)
        nrm.nrm_sync_status()
        want, want_lse, p, size, spread = ref.attention(f64(self.q), self.values(0), self.values(1), self.table.numpy(),
                                                        self.lengths.numpy(), scale, window)
        n = int(self.lengths.max()) if len(self.lengths) else 0
        top = np.where(np.isfinite(want_lse), np.abs(want_lse), 0)
        D = (2 * (self.d + 16) * U + 2.0 ** -21) * size + 16 * U * (size + top)
        rel = 2 * (2 * D + 2.0 ** -21 + 2 * (n + 64) * U)
        out_rel = rel[..., None] + 2 * (n + 64) * U + (2.0 ** -11 if self.dtype == "bf16" else 2.0 ** -21)
        vmax = spread.max() if spread.size else 0.0
        lim = out_rel * spread + n * 2.0 ** -38 * vmax
        lim = lim + half_step(self.dtype) * (np.abs(want) + lim) + TINY[self.dtype]
        assert np.array_equal(np.isnan(f64(out)), np.isnan(want))
        off = np.abs(f64(out) - want)
        assert not (off > lim).any(), (off.max(), (off / np.maximum(lim, 1e-300)).max())
        assert np.array_equal(np.isneginf(f64(lse)), np.isneginf(want_lse))
        fine = np.isfinite(want_lse)
        off = np.abs(f64(lse)[fine] - want_lse[fine])
        assert (off <= (rel + 4 * U * top)[fine]).all(), off.max()
        if weights:
            heads = self.hq // self.hk
            got = f64(w) - f64(before)
            r = rel.reshape(len(self.lengths), self.hk, heads).max(-1)[..., None]
            lim = r * p + 2 * U * (f64(before) + p) + heads * 2.0 ** -120
            assert (np.abs(got - p) <= lim).all(), (np.abs(got - p) / lim).max()
            assert (got[p == 0] == 0).all()
        return out


SHAPES = [
    # dtype, lengths, hq, hk, d, kind, group, page
    ("bf16", [1], 32, 8, 128, "e4m3", 128, 16),
    ("bf16", [1001], 32, 8, 128, "e4m3", 64, 16),
    ("f16", [1, 31, 32, 33, 0, 64, 65, 100], 16, 4, 128, "int8", 128, 32),
    ("f32", [300, 0, 7], 12, 12, 80, "e4m3", 80, 100),
    ("f32", [257], 8, 1, 64, "int4", 16, 8),
    ("bf16", [513, 2, 1030], 16, 1, 256, "int8", 256, 64),
    ("bf16", [700], 8, 2, 128, "int4", 32, 64),
    ("f16", [129, 40], 20, 4, 96, "int4", 48, 16),
    ("f16", [222], 6, 2, 96, "e4m3", 96, 100),
    ("f16", [222, 97], 48, 3, 160, "int8", 80, 100),
    ("f32", [222, 31], 34, 2, 128, "e4m3", 32, 16),
    ("bf16", [99, 5], 5, 5, 256, "int4", 64, 8),
    ("bf16", [50], 4, 2, 16, "int8", 16, 1),
    ("f16", [70], 4, 4, 192, "e4m3", 48, 16),
    ("f32", [70, 3], 3, 1, 48, "int4", 48, 16),
    # layouts of no whole vectors
    ("bf16", [70, 3], 6, 2, 72, "e4m3", 72, 16),
    ("f32", [45], 7, 7, 33, "int8", 11, 5),
    ("f16", [45, 80], 9, 1, 40, "int4", 8, 16),
    ("bf16", [45], 2, 1, 1, "int8", 1, 16),
    ("bf16", [45], 2, 1, 2, "int4", 2, 16),
    ("f16", [64, 64], 12, 2, 250, "e4m3", 125, 16),
]


@pytest.mark.parametrize("dtype,lengths,hq,hk,d,kind,group,page", SHAPES)
def test_against_the_reference(dtype, lengths, hq, hk, d, kind, group, page):
    Case(dtype, lengths, hq, hk, d, kind, group, page).check()


@pytest.mark.parametrize("dtype,lengths,hq,hk,d,kind,group,page", SHAPES)
@pytest.mark.parametrize("window", [0, 1, 33])
def test_weights_and_windows(dtype, lengths, hq, hk, d, kind, group, page, window):
    Case(dtype, lengths, hq, hk, d, kind, group, page, seed=1, loud=3.0).check(window=window, weights=True)


@pytest.mark.parametrize("order", ["pshd", "phsd", "hpsd"])
@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("kind", ["e4m3", "int8", "int4"])
def test_layouts_of_the_cache(order, offset, kind):
    Case("bf16", [65, 130], 8, 2, 64, kind, 32, 16, order=order, offset=offset).check(weights=True)


def test_many_sequences_are_cut_into_launches():
    lengths = [(7 * i) % 41 for i in range(2500)]
    c = Case("bf16", lengths, 2, 1, 32, "int8", 32, 8, width=6)
    c.check(weights=True)


def test_a_ragged_batch_and_its_sequences_alone_agree():
    # the cut of the work changes with the batch, so sums may be added in another order, no more
    lengths = [1, 2000, 0, 333, 4000, 64]
    c = Case("f32", lengths, 8, 2, 64, "e4m3", 32, 16)
    c.check(weights=True)
    c.check(window=500)


def test_the_same_call_gives_the_same_bits():
    c = Case("bf16", [777, 3000, 12], 32, 8, 128, "e4m3", 128, 16)
    w = [torch.zeros(3, 8, 3008, device="cuda") for _ in range(2)]
    a, la = c.run(weights=w[0], lse=True)
    b, lb = c.run(weights=w[1], lse=True)
    assert same(a, b) and same(la, lb) and same(*w)


def test_strided_queries_and_outputs():
    c = Case("bf16", [200, 3], 8, 2, 64, "int8", 64, 16)
    want, _ = c.run()
    qkv = torch.zeros(2, 12, 64, dtype=torch.bfloat16, device="cuda")
    qkv[:, 2:10] = c.q.cuda()
    o = torch.zeros(2, 8, 100, dtype=torch.bfloat16, device="cuda")
    got, _ = c.run(q=qkv[:, 2:10], out=o[..., :64])
    assert same(got.contiguous(), want) and not o[..., 64:].any()
    o = torch.zeros(8, 2, 65, dtype=torch.bfloat16, device="cuda")
    got, _ = c.run(q=qkv[:, 2:10], out=o.transpose(0, 1)[..., 1:])
    assert same(got.contiguous(), want) and not o[..., 0].any()


def test_batch_of_one_token_each():
    # [batch, 1, heads, d] is [sequences, heads, d] too
    c = Case("bf16", [200, 3], 8, 2, 64, "int8", 64, 16)
    want, _ = c.run()
    out = torch.empty(2, 1, 8, 64, dtype=torch.bfloat16, device="cuda")
    got, _ = c.run(q=c.q.cuda().unsqueeze(1), out=out)
    assert same(got.view(2, 8, 64), want)


@pytest.mark.parametrize("kind", ["e4m3", "int8", "int4"])
@pytest.mark.parametrize("d", [64, 40])
def test_poison_outside_the_sequence_stays_out(kind, d):
    group = 16 if d == 64 else 8
    clean = Case("f32", [45, 0, 17], 4, 2, d, kind, group, 16, poison=0.0).run(window=20)[0]
    for poison in (float("nan"), float("inf"), -3e38):
        assert same(Case("f32", [45, 0, 17], 4, 2, d, kind, group, 16, poison=poison).run(window=20)[0], clean)


@pytest.mark.parametrize("d,kind", [(64, "e4m3"), (64, "int8"), (64, "int4"), (40, "e4m3")])
def test_a_nan_row_reaches_the_heads_that_read_it(d, kind):
    c = Case("f32", [45, 33], 4, 2, d, kind, d, 16)
    # position 20 of sequence 0, head 1 of the keys: its queries are NaN, all others as before
    want, _ = c.run()
    c.scales[0][c.table[0, 1], 4, 1] = float("nan")
    got, lse = c.run(lse=True)
    assert got[0, 2:].isnan().all() and lse[0, 2:].isnan().all()
    assert same(got[0, :2], want[0, :2]) and same(got[1], want[1])
    c.scales[0][c.table[0, 1], 4, 1] = 0.01
    c.scales[1][c.table[0, 1], 4, 1] = float("nan")
    got, lse = c.run(lse=True)
    assert got[0, 2:].isnan().all() and not lse.isnan().any() and not got[0, :2].isnan().any()


@pytest.mark.parametrize("d", [64, 40])
def test_rows_of_zeros_and_equal_logits(d):
    # all codes 0: the mean of zeros; equal keys: the mean of the values
    c = Case("f32", [100], 4, 2, d, "int8", d, 16)
    c.scales[0].zero_()
    _, lse = c.run(lse=True)
    assert np.allclose(f64(lse), np.log(100), rtol=8 * U, atol=0)
    c.check()
    c.scales[1].zero_()
    out, _ = c.run()
    assert not out.any()


@pytest.mark.parametrize("d", [64, 40])
@pytest.mark.parametrize("loud", [1e-30, 1.0, 60.0])
def test_small_and_large_logits(d, loud):
    Case("f32", [300, 40], 4, 2, d, "e4m3", d, 16, loud=loud).check(weights=True)
    Case("bf16", [300, 40], 4, 2, d, "int8", d, 16, loud=loud).check()


def test_scales_of_values_over_the_whole_range():
    # values of very different sizes: each output channel's group keeps its own precision
    for d, group in ((64, 16), (40, 8)):
        c = Case("f32", [90], 4, 2, d, "e4m3", group, 16, poison=0.0)
        c.scales[1].mul_(torch.logspace(-18, 12, c.scales[1].shape[-1], device="cuda"))
        c.check()
        c.scales[1].mul_(1e-25)
        c.check()


@pytest.mark.parametrize("d", [64, 40])
@pytest.mark.parametrize("kind", ["e4m3", "int8", "int4"])
def test_negative_scales(d, kind):
    # a cache that something else has written may hold them
    c = Case("f32", [90, 33, 1], 4, 2, d, kind, 8 if d == 40 else 16, 16)
    for t in range(2):
        c.scales[t][:, ::2] *= -3
    c.check(weights=True)
    c.scales[1].abs_().neg_()
    c.check()


@pytest.mark.parametrize("d", [64, 40])
def test_lengths_and_pages_out_of_range_are_reported(d):
    c = Case("f32", [45, 60, 30], 4, 2, d, "int8", d, 16, width=4, poison=0.0)
    good, _ = c.run()
    nrm.nrm_sync_status()
    table = c.table.clone()
    c.lengths = torch.tensor([-5, 65, 30])
    out, lse = c.run(lse=True)
    with pytest.raises(nrm.NrmError) as e:
        nrm.nrm_sync_status()
    assert e.value.status == nrm.NRM_ERR_INVALID_ARG
    assert not out[0].any() and lse[0].isneginf().all() and same(out[2], good[2])
    c.lengths = torch.tensor([45, 64, 30])
    assert same(c.run()[0][1], out[1])
    nrm.nrm_sync_status()
    for bad in (-1, -2 ** 62, c.cache.slots, 2 ** 62):
        # the positions of that page are left out, as if the sequence had none there
        c.lengths = torch.tensor([45, 60, 30])
        c.table = table.clone()
        c.table[0, 1] = bad
        w = torch.zeros(3, 2, 64, device="cuda")
        out, _ = c.run(weights=w)
        with pytest.raises(nrm.NrmError):
            nrm.nrm_sync_status()
        want = ref.attention(f64(c.q), c.values(0), c.values(1), c.table.numpy(), c.lengths.numpy(), d ** -0.5)[0]
        assert np.allclose(f64(out), want, rtol=1e-4, atol=1e-5)
        assert not w[0, :, 16:32].any() and w[0, :, :16].all()
        # entries behind the last position are not read
        c.table = table.clone()
        c.table[0, 3] = c.table[2, 2:] = bad
        assert same(c.run()[0], good)
        nrm.nrm_sync_status()


def test_a_length_above_the_weights_is_out_of_range():
    c = Case("f32", [45, 60], 4, 2, 64, "int8", 64, 16)
    w = torch.zeros(2, 2, 50, device="cuda")
    c.run(weights=w)
    with pytest.raises(nrm.NrmError):
        nrm.nrm_sync_status()


def test_shared_pages_and_a_view_of_the_weights():
    # two sequences begin with the same pages; the weights are rows of a larger tensor
    c = Case("f32", [60, 60], 4, 2, 64, "int8", 64, 16)
    c.table[1, :2] = c.table[0, :2]
    pool = torch.zeros(2, 3, 100, device="cuda")
    c.run(weights=pool[:, 1:, 20:84])
    w = torch.zeros(2, 2, 64, device="cuda")
    c.run(weights=w)
    assert same(pool[:, 1:, 20:84].contiguous(), w)
    assert not pool[:, 0].any() and not pool[..., :20].any() and not pool[..., 84:].any()
    c.check(weights=True)


def test_no_sequences_and_no_positions():
    c = Case("bf16", [5], 4, 2, 64, "int8", 64, 16)
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    ws = nrm.kv_attention_workspace(e, c.cache, c.table[:0])
    nrm.nrm_kv_cache_attention(e, c.cache, c.table[:0].cuda(), c.lengths[:0].cuda(), e.clone(), 1.0, ws)
    c.lengths = torch.tensor([0])
    out, lse = c.run(lse=True)
    assert not out.any() and lse.isneginf().all()
    nrm.nrm_sync_status()


@pytest.mark.parametrize("d", [64, 40])
def test_far_offsets(d):
    # pages more than 2^31 bytes apart
    kind = torch.int8
    big = torch.zeros((3 << 30) + 4096, dtype=kind, device="cuda")
    codes = [torch.as_strided(big, (3, 16, 2, d), (3 << 29, 2 * d, d, 1), t * 2048) for t in range(2)]
    g = torch.Generator(device="cuda").manual_seed(0)
    for t in codes:
        t.copy_(torch.randint(-127, 128, t.shape, generator=g, device="cuda"))
    scales = [torch.rand(3, 16, 2, 1, generator=g, device="cuda") / 60 for _ in range(2)]
    cache = nrm.kv_cache(codes[0], scales[0], codes[1], scales[1])
    near = nrm.kv_cache(codes[0].contiguous(), scales[0], codes[1].contiguous(), scales[1])
    q = torch.randn(1, 8, d, generator=g, device="cuda")
    table, n = torch.tensor([[2, 0, 1]], device="cuda"), torch.tensor([41], device="cuda")
    ws, outs = nrm.kv_attention_workspace(q, cache, table), []
    for c in (cache, near):
        outs.append(torch.empty_like(q))
        nrm.nrm_kv_cache_attention(q, c, table, n, outs[-1], 0.1, ws)
    assert same(*outs)


@pytest.mark.parametrize("kind", ["e4m3", "int4"])
def test_strides_beyond_32_bits_of_vectors(kind):
    # a cache described as spanning more than 2^36 bytes, of which the sequence uses the first page
    c = Case("bf16", [60], 8, 2, 128, kind, 32, 64)
    want, _ = c.run()
    far = c.cache._c
    page = int(c.table[0, 0])
    for name, step in (("k_codes", c.codes[0].stride(0)), ("v_codes", c.codes[1].stride(0)), ("k_scales", 4 * c.scales[0].stride(0)),
                       ("v_scales", 4 * c.scales[1].stride(0))):
        setattr(far, name, getattr(far, name) + page * step)
    far.pages, far.page_stride = 2, 1 << 38
    table = c.table.clone()
    c.table = torch.zeros_like(table)
    got, _ = c.run()
    assert same(got, want)
    nrm.nrm_sync_status()


@pytest.mark.parametrize("d,group", [(256, 32), (256, 64), (192, 64), (192, 192), (224, 32), (160, 32), (144, 48), (112, 16), (64, 64), (32, 32)])
@pytest.mark.parametrize("kind", ["e4m3", "int8", "int4"])
def test_rows_and_groups_of_every_kernel(d, group, kind):
    # whole and partial tiles, one and two eights of heads
    Case("bf16", [33, 128, 5], 10, 1, d, kind, group, 16).check(weights=True)
    Case("f32", [70], 3, 1, d, kind, group, 16).check()


def test_captured_and_replayed():
    c = Case("bf16", [300, 41], 8, 2, 64, "int8", 64, 16)
    q, table, lengths = c.q.cuda(), c.table.cuda(), c.lengths.cuda()
    out, w = torch.empty_like(q), torch.zeros(2, 2, 304, device="cuda")
    ws = nrm.kv_attention_workspace(q, c.cache, table, weights=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nrm.nrm_kv_cache_attention(q, c.cache, table, lengths, out, 0.125, ws, weights=w)
    for n in ([300, 41], [1, 304], [0, 17], [33, 32]):  # other lengths, on the device
        c.lengths = torch.tensor(n)
        lengths.copy_(c.lengths)
        q.copy_(torch.randn_like(q))
        w.zero_()
        ws.fill_(0xff)
        graph.replay()
        again = torch.zeros_like(w)
        assert same(out, c.run(q=q, weights=again, scale=0.125)[0]) and same(w, again)


def test_two_streams_with_workspaces_of_their_own():
    cases = [Case("bf16", [2000 + i, 100], 16, 4, 64, "int8", 64, 16, seed=i) for i in range(2)]
    want = [c.run()[0] for c in cases]
    q, tables, lengths = ([getattr(c, n).cuda() for c in cases] for n in ("q", "table", "lengths"))
    outs = [torch.empty_like(x) for x in q]
    ws = [nrm.kv_attention_workspace(q[i], c.cache, tables[i]) for i, c in enumerate(cases)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(50):
        for i, c in enumerate(cases):
            nrm.nrm_kv_cache_attention(q[i], c.cache, tables[i], lengths[i], outs[i], 64 ** -0.5, ws[i], stream=streams[i])
    torch.cuda.synchronize()
    assert same(outs[0], want[0]) and same(outs[1], want[1])


@pytest.mark.parametrize("seed", range(40))
def test_random_shapes(seed):
    rng = np.random.default_rng(seed)
    d = int(rng.choice([16, 32, 48, 64, 80, 96, 112, 128, 160, 192, 208, 256, 24, 100, int(rng.integers(1, 257))]))
    kind = str(rng.choice(["e4m3", "int8", "int4"]))
    if kind == "int4":
        d += d % 2
    groups = [g for g in range(1, d + 1) if d % g == 0 and (kind != "int4" or g % 2 == 0)]
    group = int(rng.choice([g for g in groups if g % 16 == 0] or groups)) if rng.random() < 0.7 else int(rng.choice(groups))
    hk = int(rng.integers(1, 6))
    hq = hk * int(rng.choice([1, 2, 3, 4, 5, 8, 9, 16, 17, 33]))
    lengths = [int(rng.choice([0, 1, rng.integers(1, 40), rng.integers(1, 700)])) for _ in range(int(rng.integers(1, 7)))]
    c = Case(str(rng.choice(["bf16", "f16", "f32"])), lengths, hq, hk, d, kind, group, int(rng.choice([1, 5, 8, 16, 64, 100])),
             seed=seed, order=str(rng.choice(["pshd", "phsd"])), loud=float(rng.choice([0.1, 1, 4])))
    c.check(window=int(rng.choice([0, 0, rng.integers(1, 300)])), weights=bool(rng.random() < 0.5))
