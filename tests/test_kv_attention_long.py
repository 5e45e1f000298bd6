"""Attention over the paged cache in pieces of a thousand tiles for each worker, where what is off a
little in each tile adds up, against the double-precision reference (oracle/served.py).

Tolerances, derived before the first run.  u = 2^-24 is half a step of float32.
  * A logit l_j: float32 sums of d products in any order, 2u each, of factors with 22 bits for
    float32 queries (2^-21); scale, key's scale, and base 2 and back: 16 u (|l_j| + |lse|).
    D_j = (2 (d + 16) u + 2^-21) S_j + 16 u (|l_j| + |lse|), S_j = scale sum |q k_j|.  Where queries are
    +-c, c of few bits, and the codes whole numbers, all sums are exact: the first part is 0.
  * p_j = 2^(l_j - m): 2 D_j, the function's 2^-21 and the sum's (2 N + 64) u, N the tiles of a piece
    (a tile's positions are added in a few levels, the tiles in turn), for p_j and for the sum.
  * A weight: p_j times its value's scale, rounded to 22 bits (2^-22; bfloat16 11, 2^-11), of which
    what is below 2^-50 (bfloat16 2^-39) of the largest p_j times the largest scale may be lost.
  * out: a tile's products reach a sum in up to 4 additions (two halves, two factors), each cut off at
    4 u of what it holds: (16 N + 64) u of sum p |v|.  Then half a step of the type.
"""
import numpy as np
import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
from oracle import served as ref
from test_heads import DT, TINY, U, f64, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    nrm.load()


def parts(codes, scales, kind):
    """Codes as numbers and the scales of their elements, [positions, d]."""
    x = ref.stored(codes, np.ones_like(scales), kind)
    return x, np.repeat(scales.astype(np.float64), x.shape[-1] // scales.shape[-1], -1)


def check_rows(dtype, kind, q, k, v, scale, out, lse, tiles, exact=()):
    """One sequence's heads on one head of the keys.  q, out [heads, d], lse [heads]; k, v: (codes, scales) of the
    positions; `exact`: positions whose logits' sums are exact."""
    (kc, ks), (vc, vs) = parts(*k, kind), parts(*v, kind)
    d = q.shape[1]
    for h in range(q.shape[0]):
        l = scale * (kc * ks) @ q[h]
        want_lse = l.max() + np.log(np.exp(l - l.max()).sum())
        p = np.exp(l - want_lse)
        S = scale * np.abs(kc * ks) @ np.abs(q[h])
        D = (2 * (d + 16) * U + 2.0 ** -21) * S
        D[list(exact)] = 0
        D = D + 16 * U * (np.abs(l) + abs(want_lse))
        add = (2 * tiles + 64) * U
        mean = (p * D).sum()  # of the sum
        rel = 2 * (D + mean) + 2.0 ** -20 + 2 * add
        bf16 = dtype == "bf16"
        want = p @ (vc * vs)
        lim = (p * (rel + (2.0 ** -11 if bf16 else 2.0 ** -22))) @ np.abs(vc * vs)
        lim = lim + 2.0 ** (-39 if bf16 else -50) * p.max() * np.abs(vs).max(0) * np.abs(vc).sum(0)
        lim = lim + (16 * tiles + 64) * U * (p @ np.abs(vc * vs))
        lim = lim + half_step(dtype) * (np.abs(want) + lim) + TINY[dtype]
        off = np.abs(out[h] - want)
        assert (off <= lim).all(), (h, off.max(), np.abs(want).max(), (off / lim).max())
        assert abs(lse[h] - want_lse) <= 2 * mean + 2.0 ** -20 + add + 4 * U * abs(want_lse), (h, lse[h], want_lse)


class Long:
    """Sequences that share the pages of one, in their own order, as many as give each worker a piece of a
    thousand tiles."""

    def __init__(self, dtype, kind, lower, positions=32768, seqs=64, hk=32, d=64, page=64, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.page, self.hk, self.d, self.kind, self.dtype = page, hk, d, kind, dtype
        pages = positions // page
        self.sign = torch.where(torch.randn(d, generator=g) > 0, 1.0, -1.0)
        # keys: -sign times a number near 1, quantised; queries: sign times a few sizes.  Logits in base 2 about `lower`.
        near = 1 + 0.02 * torch.randn(pages, page, hk, 1, generator=g) + 0.05 * torch.randn(pages, page, hk, d, generator=g)
        top = {"e4m3": 240, "int8": 100}[kind]
        codes = -self.sign * near * top
        self.kc = codes.to(torch.float8_e4m3fn) if kind == "e4m3" else codes.round().clamp(-127, 127).to(torch.int8)
        self.ks = torch.full((pages, page, hk, 1), 1 / top)
        vals = torch.randn(pages, page, hk, d, generator=g).abs() * top / 4
        self.vc = vals.to(torch.float8_e4m3fn) if kind == "e4m3" else vals.round().clamp(-127, 127).to(torch.int8)
        self.vs = torch.rand(pages, page, hk, 1, generator=g) / top
        self.table = torch.stack([torch.arange(pages) if s % 2 == 0 else torch.arange(pages).flip(0) for s in range(seqs)])
        self.lengths = torch.full((seqs,), positions)
        # scale 1, in base 2: -|q| d log2(e)
        size = torch.tensor(lower).repeat(-(-seqs // len(lower)))[:seqs] / (d * 1.4426950408889634)
        self.q = (size[:, None, None] * self.sign * (1 + 0.01 * torch.rand(seqs, hk, 1, generator=g))).to(DT[dtype])

    def run(self):
        cache = nrm.kv_cache(*(t.cuda() for t in (self.kc, self.ks, self.vc, self.vs)))
        q, table, n = self.q.cuda(), self.table.cuda(), self.lengths.cuda()
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        w = torch.zeros(len(n), self.hk, self.table.shape[1] * self.page, device="cuda")
        nrm.nrm_kv_cache_attention(q, cache, table, n, out, 1.0, nrm.kv_attention_workspace(q, cache, table, weights=True), lse=lse,
                                   weights=w)
        nrm.nrm_sync_status()
        return out, lse, w

    def check(self, out, lse, seqs):
        for s in seqs:
            j = np.arange(int(self.lengths[s]))
            at = (self.table[s, j // self.page], j % self.page)
            for h in (0, 13, self.hk - 1):
                codes = [t.view(torch.uint8)[at[0], at[1], h].view(t.dtype).float().numpy() for t in (self.kc, self.vc)]
                scales = [t[at[0], at[1], h].numpy() for t in (self.ks, self.vs)]
                check_rows(self.dtype, self.kind, f64(self.q)[s, h:h + 1], (codes[0], scales[0]), (codes[1], scales[1]), 1.0,
                           f64(out)[s, h:h + 1], f64(lse)[s, h:h + 1], len(j) // 32)


@pytest.mark.parametrize("dtype,kind", [("f32", "e4m3"), ("f32", "int8"), ("f16", "e4m3"), ("bf16", "int8")])
def test_long_pieces_of_negative_logits(dtype, kind):
    # the largest of a sequence's logits stays the same for hundreds of tiles, and is below 0
    c = Long(dtype, kind, [12.4, 28.7, 61.3, 125.9, 6.2, 254.6])
    out, lse, w = c.run()
    # each head's weights add up to 1: of the same logits as its sum, so that theirs do not count.  Half a step for
    # each of a piece's additions and of the exponents' parts, twice the function's
    lim = (2 * 1024 + 64) * U + 16 * U * 260 + 2.0 ** -20
    total = w.double().sum(-1)
    assert float((total - 1).abs().max()) <= lim, (float((total - 1).abs().max()), lim)
    c.check(out, lse, range(6))


@pytest.mark.parametrize("dtype,kind", [("f32", "int8"), ("f16", "e4m3"), ("bf16", "e4m3"), ("bf16", "int8")])
def test_long_pieces_whose_largest_numbers_come_first_or_last(dtype, kind):
    # even sequences meet ever larger logits and values, odd ones ever smaller ones
    c = Long(dtype, kind, [20.0, 20.0, 3.0, 3.0], seed=1)
    pages = c.ks.shape[0]
    c.ks *= torch.linspace(1.5, 0.5, pages)[:, None, None, None]
    c.vs *= torch.logspace(-12, 6, pages)[:, None, None, None]
    out, lse, w = c.run()
    c.check(out, lse, range(4))
    c.vs = c.vs.flip(0)
    out, lse, w = c.run()
    c.check(out, lse, range(4))
