"""Eviction from the paged cache by weight, against the reference (oracle/served.py): whole
numbers and copies, so everything is equal, bit for bit."""
import numpy as np
import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
from oracle import served as ref
from test_kv_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    nrm.load()


def raw(t):
    return t.contiguous().view(torch.uint8)


class Evict:
    def __init__(self, lengths, keep, hk=2, d=64, kind="int8", group=None, page=16, first=0, recent=0, seed=0, order="pshd",
                 offset=0, weights=None):
        self.c = Case("bf16", [*lengths, *([keep] * len(lengths))], hk, hk, d, kind, group, page, seed=seed, order=order,
                      offset=offset, poison=1.0)
        n = len(lengths)
        self.table, self.new_table = self.c.table[:n].cuda(), self.c.table[n:, :-(-keep // page)].cuda()
        self.lengths = torch.tensor(lengths).cuda()
        self.cap, self.keep, self.first, self.recent, self.hk, self.page = self.table.shape[1] * page, keep, first, recent, hk, page
        g = torch.Generator().manual_seed(seed)
        w = torch.rand(n, hk, self.cap, generator=g)
        # zeros, equal ones, and numbers of every size
        w = torch.where(torch.rand(w.shape, generator=g) < 0.2, 0.0, w * 2.0 ** torch.randint(-140, 100, w.shape, generator=g))
        w = torch.where(torch.rand(w.shape, generator=g) < 0.2, 0.25, w)
        self.weights = w.cuda() if weights is None else weights
        self.new_lengths = torch.full((n,), -7, device="cuda")
        self.new_weights = torch.full((n, hk, keep + 3), 9.0, device="cuda")
        self.kept = torch.full((n, hk, keep), -7, device="cuda")

    def run(self, stream=None):
        nrm.nrm_kv_cache_evict(self.c.cache, self.table, self.lengths, self.weights, self.new_table, self.new_lengths,
                               self.new_weights, self.kept, first=self.first, recent=self.recent, stream=stream)

    def check(self):
        before = [(raw(self.c.codes[t]).cpu().clone(), self.c.scales[t].cpu().clone()) for t in range(2)]
        self.run()
        nrm.nrm_sync_status()
        w = self.weights.cpu().numpy()
        kept, new = ref.evict(w, self.lengths.cpu().numpy(), self.keep, self.first, self.recent, self.cap)
        assert np.array_equal(self.kept.cpu().numpy(), kept)
        assert np.array_equal(self.new_lengths.cpu().numpy(), new)
        got = self.new_weights.cpu().numpy()
        table, new_table = self.table.cpu().numpy(), self.new_table.cpu().numpy()
        for t in range(2):
            codes = before[t][0].view(*self.c.codes[t].shape[:3], -1).numpy().copy()
            scales = before[t][1].numpy().copy()
            page = self.page
            for s in range(len(new)):
                for h in range(self.hk):
                    j, i = kept[s, h, :new[s]], np.arange(new[s])
                    assert np.array_equal(got[s, h, :new[s]], w[s, h, j], equal_nan=True)
                    assert (got[s, h, new[s]:] == 9.0).all()
                    src = (table[s, j // page], j % page, h)
                    dst = (new_table[s, i // page], i % page, h)
                    codes[dst], scales[dst] = codes[src], scales[src]
            assert np.array_equal(raw(self.c.codes[t]).cpu().view(codes.shape).numpy(), codes)
            assert np.array_equal(self.c.scales[t].cpu().numpy().view(np.uint32), scales.view(np.uint32))


@pytest.mark.parametrize("lengths,keep,first,recent", [
    ([100], 40, 0, 0), ([100], 40, 4, 10), ([100], 40, 40, 0), ([100], 40, 0, 40), ([100], 40, 17, 23), ([100], 1, 0, 0),
    ([100], 1, 1, 0), ([100], 99, 0, 0), ([100], 100, 3, 3), ([0, 1, 39, 40, 41, 3000], 40, 2, 5), ([5000], 2500, 4, 100),
    ([1025, 1024, 2049], 1024, 0, 1), ([33], 32, 0, 0),
    # on both sides of what a CTA ranks at once
    ([256, 0, 255, 3], 128, 3, 60), ([257, 256, 2], 129, 3, 60), ([2, 1, 0], 1, 0, 0), ([256], 255, 0, 0), ([256], 1, 0, 0),
])
def test_against_the_reference(lengths, keep, first, recent):
    Evict(lengths, keep, first=first, recent=recent).check()


@pytest.mark.parametrize("kind,d,group,page,order,offset", [
    ("e4m3", 128, 32, 16, "pshd", 0), ("e4m3", 80, 80, 100, "phsd", 0), ("int4", 128, 32, 32, "pshd", 0),
    ("int4", 40, 8, 16, "pshd", 0), ("int4", 2, 2, 1, "pshd", 0), ("int8", 33, 11, 5, "hpsd", 0), ("int8", 256, 16, 8, "pshd", 0),
    ("e4m3", 64, 64, 16, "pshd", 1), ("int8", 64, 16, 16, "pshd", 8), ("int8", 1, 1, 16, "pshd", 0), ("int8", 72, 8, 16, "pshd", 4),
])
def test_layouts_of_the_cache(kind, d, group, page, order, offset):
    Evict([200, 7, 90], 50, 3, d, kind, group, page, 1, 9, order=order, offset=offset).check()


@pytest.mark.parametrize("values", [
    [0.0, -0.0], [float("nan"), 1.0, float("inf")], [-1.0, -2.0, 0.0, 3.0, -float("inf")],
    [1.0, 1.0 + 2 ** -23, 1.0 - 2 ** -24], [2.0 ** -149, 0.0, 2.0 ** -126], [3.4e38, 3.3e38],
])
def test_ties_and_special_weights(values):
    g = torch.Generator().manual_seed(len(values))
    for n, keep in ((100, 37), (2100, 1000)):
        e = Evict([n], keep, first=1, recent=2)
        e.weights.copy_(torch.tensor(values)[torch.randint(0, len(values), e.weights.shape, generator=g)])
        e.check()


def test_without_new_weights_and_with_views():
    e = Evict([100, 60], 40, first=2, recent=3)
    pool = torch.zeros(2, 5, 200, device="cuda")
    pool[:, 1:5:2, 10:10 + e.cap] = e.weights
    kept, new = ref.evict(e.weights.cpu().numpy(), [100, 60], 40, 2, 3, e.cap)
    e.weights, e.new_weights = pool[:, 1:5:2, 10:10 + e.cap], None
    wide = torch.full((2, 9), -1, device="cuda")
    wide[:, 2:2 + e.new_table.shape[1]] = e.new_table
    e.new_table = wide[:, 2:2 + e.new_table.shape[1]]
    e.run()
    nrm.nrm_sync_status()
    assert np.array_equal(e.kept.cpu().numpy(), kept)


def test_lengths_and_pages_out_of_range_are_reported():
    e = Evict([100, 60, 90], 40)
    e.lengths.copy_(torch.tensor([-3, 10 ** 6, 90]))
    e.run()
    with pytest.raises(nrm.NrmError) as err:
        nrm.nrm_sync_status()
    assert err.value.status == nrm.NRM_ERR_INVALID_ARG
    assert e.new_lengths.tolist() == [0, 40, 40] and (e.kept[0] == -1).all()
    kept, _ = ref.evict(e.weights.cpu().numpy(), [0, e.cap, 90], 40, 0, 0, e.cap)
    assert np.array_equal(e.kept.cpu().numpy(), kept)
    for bad in (-1, -2 ** 62, e.c.cache.slots, 2 ** 62):
        for which in ("table", "new_table"):
            e = Evict([100], 40)
            getattr(e, which)[0, 1] = bad
            before = [raw(t).cpu().clone() for t in (*e.c.codes, *e.c.scales)]
            e.run()
            with pytest.raises(nrm.NrmError):
                nrm.nrm_sync_status()
            # the rows on good pages were copied, nothing else was touched
            for t in range(2):
                want = before[t].view(e.c.codes[t].shape).clone()
                old, new = e.table.cpu(), e.new_table.cpu()
                for h in range(2):
                    for i, j in enumerate(e.kept[0, h].tolist()):
                        a, b = int(old[0, j // 16]), int(new[0, i // 16])
                        if bad not in (a, b):
                            want[b, i % 16, h] = before[t].view(want.shape)[a, j % 16, h]
                assert torch.equal(raw(e.c.codes[t]).cpu().view(want.shape), want)


def test_captured_and_replayed():
    e = Evict([300, 200], 64, first=1, recent=7)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e.run()
    for n in ([300, 200], [64, 65], [1, 0]):
        e.lengths.copy_(torch.tensor(n))
        e.weights.copy_(torch.rand_like(e.weights))
        e.kept.fill_(-7)
        graph.replay()
        nrm.nrm_sync_status()
        kept, new = ref.evict(e.weights.cpu().numpy(), n, 64, 1, 7, e.cap)
        assert np.array_equal(e.kept.cpu().numpy(), kept) and e.new_lengths.tolist() == new.tolist()


@pytest.mark.parametrize("seed", range(25))
def test_random_shapes(seed):
    rng = np.random.default_rng(seed)
    kind = str(rng.choice(["e4m3", "int8", "int4"]))
    d = 2 * int(rng.integers(1, 129)) if rng.random() < 0.4 else int(rng.choice([64, 80, 96, 128, 256]))
    groups = [g for g in range(1, d + 1) if d % g == 0 and (kind != "int4" or g % 2 == 0)]
    lengths = [int(rng.choice([0, rng.integers(1, 60), rng.integers(1, 4000)])) for _ in range(int(rng.integers(1, 6)))]
    keep = int(rng.integers(1, max(2, max(lengths))))
    first = int(rng.integers(0, keep + 1))
    recent = int(rng.integers(0, keep - first + 1))
    if rng.random() < 0.6:
        first, recent = first // 4, recent // 4
    Evict(lengths, keep, int(rng.integers(1, 5)), d, kind, int(rng.choice(groups)), int(rng.choice([1, 8, 16, 100])), first, recent,
          seed=seed, order=str(rng.choice(["pshd", "phsd"]))).check()
