"""Eviction of sequences so long that a cluster of CTAs chooses for each head, or that their weights do
not stay in shared memory: exact, as the shorter ones."""
import numpy as np
import pytest
import torch

from oracle import served as ref
from test_kv_evict import Evict, _gpu  # noqa: F401

pytestmark = pytest.mark.gpu

# One CTA for each 8192 positions up to 8, as powers of two, while twice as many fill no more than two waves; a CTA
# holds 46080 weights.  152 SMs: 152 heads at most get two CTAs, 76 four and 38 eight.
CASES = [
    # lengths (the first the longest), keep, heads of keys, first, recent
    ([8193], 4000, 2, 0, 0),
    ([8193, 8192, 4097, 4096, 2049, 3, 0], 2048, 3, 5, 7),
    ([16384, 16385, 9000, 8192, 100], 8192, 2, 4100, 100),       # `first` ends in the second CTA's part
    ([20000, 10001, 20000], 9000, 2, 2, 6000),                   # `recent` begins in the second to last one's
    ([40000, 8193, 33000, 2500, 0], 2500, 2, 0, 2500),           # nothing between is taken
    ([40000, 39999, 4000], 39998, 1, 1, 1),
    ([70001, 70000, 10240, 10241, 1], 10240, 2, 10, 64),         # some CTAs of the shorter have no position
    ([70001, 65536], 1, 2, 0, 0),
    ([70001], 60000, 1, 20000, 20000),
    # not held: eight CTAs, then four, then one
    ([46080 * 8 + 2049, 5000], 100000, 1, 3, 9),
    ([46080 * 4 + 1, 46080 * 4 - 5000, 100, 7, 0], 30000, 8, 3, 9),
    ([46081, 100, 46080, *([50] * 17)], 64, 8, 3, 9),
]


def few_values(e, seed):
    """Weights of so few values that the border's ties lie in every CTA's part."""
    g = torch.Generator().manual_seed(seed)
    values = torch.tensor([0.0, 0.25, 0.25 + 2.0 ** -25, 0.5, float("inf"), -1.0])
    share = torch.tensor([0.2, 0.3, 0.2, 0.2, 0.02, 0.08]).cumsum(0)
    e.weights.copy_(values[torch.searchsorted(share, torch.rand(e.weights.shape, generator=g)).clamp(max=5)])
    return e


# weights of every size too, where there are no more than two million of them
KINDS = [(*c, ties) for c in CASES for ties in ("few", "equal", "any")
         if ties != "any" or len(c[0]) * c[2] * max(c[0]) <= 2_000_000]


@pytest.mark.parametrize("lengths,keep,heads,first,recent,ties", KINDS)
def test_long_sequences(lengths, keep, heads, first, recent, ties, monkeypatch):
    monkeypatch.setattr(ref, "evict", ranked)
    e = Evict(lengths, keep, heads, 2, "int8", 2, 16, first, recent)
    if ties == "few":
        few_values(e, keep)
    elif ties == "equal":
        e.weights.fill_(1.0)
    e.check()


def ranked(weights, lengths, keep, first, recent, cap):
    """oracle.served.evict, by one sort of a head's positions."""
    seqs, heads = weights.shape[:2]
    kept, new = np.full((seqs, heads, keep), -1, dtype=np.int64), np.zeros(seqs, dtype=np.int64)
    for s in range(seqs):
        n = min(max(int(lengths[s]), 0), cap)
        new[s] = min(n, keep)
        for h in range(heads):
            if n <= keep:
                kept[s, h, :n] = np.arange(n)
                continue
            w = weights[s, h, first:n - recent].astype(np.float64)
            order = np.lexsort((np.arange(len(w)), -np.where(np.isnan(w), 0, w), ~np.isnan(w)))
            best = first + order[:keep - first - recent]
            kept[s, h] = np.sort(np.concatenate([np.arange(first), best, np.arange(n - recent, n)]))
    return kept, new


def test_the_sort_ranks_as_the_reference():
    g = np.random.default_rng(0)
    w = g.choice([0.0, -0.0, 1.0, 2.0, np.nan, np.inf, -np.inf, -3.0], (2, 2, 60)).astype(np.float32)
    for got, want in zip(ranked(w, [60, 31], 30, 3, 4, 60), ref.evict(w, [60, 31], 30, 3, 4, 60)):
        assert np.array_equal(got, want)


def test_captured_and_replayed_beside_another():
    # two clusters' calls on streams of their own, captured into one graph; other lengths and weights at each replay
    cases = [Evict([20000, 9000], 4000, 2, 16, "int8", 16, 16, 3, 50, seed=i) for i in range(2)]
    for e in cases:
        e.run()  # (the kernels are loaded)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        cases[0].run()
        cases[1].run(stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for n in ([20000, 9000], [8193, 20000], [4000, 4001], [0, 16385]):
        for e in cases:
            e.lengths.copy_(torch.tensor(n))
            e.weights.copy_(torch.rand_like(e.weights))
            e.kept.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        for e in cases:
            kept, new = ranked(e.weights.cpu().numpy(), n, 4000, 3, 50, e.cap)
            assert np.array_equal(e.kept.cpu().numpy(), kept) and e.new_lengths.tolist() == new.tolist()
