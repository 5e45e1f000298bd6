"""The angles of the rotation against products reduced exactly, to the bound that the header states.

The pair (1, 0) turned is (cos, sin) itself.  The angle is off by at most 2^-28 + 2^-32 + |pos| * 2^-61
turns, and cosine and sine, taken within an eighth of a turn, by one unit in the last place, 2^-24 at
most there: together less than 1.5 * 2^-24 at near positions."""
import numpy as np
import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
from oracle import heads as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    nrm.load()


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("offset", [0, 1])  # vectors, and element by element
@pytest.mark.parametrize("far", [0, 1 << 31, -(1 << 33), 1 << 36])
def test_cosines_and_sines_to_the_stated_bound(far, offset, inverse):
    tokens, rot = 64, 256
    rng = np.random.default_rng(abs(far) % 1000 + offset)
    pos = torch.from_numpy(rng.integers(-5000, 5000, tokens)).cuda() + far
    # frequencies of every size, 2 pi among them; the last ones turn by about half a turn at a position
    inv = np.concatenate([2 * np.pi * 10.0 ** -rng.uniform(0, 6, 96), np.pi * (1 + rng.uniform(-1e-3, 1e-3, 32))])
    inv = torch.from_numpy(np.minimum(inv, 2 * np.pi).astype(np.float32)).cuda()
    buf = torch.zeros(tokens * rot + offset, device="cuda")
    q = buf[offset:].view(tokens, 1, rot)
    q[..., :rot // 2] = 1
    out = torch.empty_like(buf)[offset:].view(tokens, 1, rot)
    (nrm.nrm_rope_bwd if inverse else nrm.nrm_rope_fwd)(q, None, pos, inv, out, None)
    a = ref.angles(pos.cpu().numpy(), inv.cpu().numpy())
    want = np.concatenate([np.cos(a), np.sin(a) * (-1.0 if inverse else 1.0)], 1)[:, None]
    off = 2 * np.pi * (2.0 ** -28 + 2.0 ** -32 + (abs(far) + 5000) * 2.0 ** -61)
    assert np.abs(out.double().cpu().numpy() - want).max() <= off + 2.0 ** -24 + 1e-15


def test_whole_quarter_turns_are_exact():
    # a frequency of pi / 2 in float32 is 2^-26.6 turns off a quarter turn, which a few positions keep far below
    # half a step of 1: cosines and sines of 0, 1, 2, ... quarter turns, either way
    pos = torch.arange(-8, 9, device="cuda")
    q = torch.zeros(17, 1, 2, device="cuda")
    q[..., 0] = 1
    out = torch.empty_like(q)
    inv = torch.full((1,), np.pi / 2, device="cuda")
    nrm.nrm_rope_fwd(q, None, pos, inv, out, None)
    n = pos.cpu().numpy()
    want = np.stack([np.array([1, 0, -1, 0])[n % 4], np.array([0, 1, 0, -1])[n % 4]], 1)
    # (the frequency itself is off by 4.4e-8 of a turn's radians a position)
    assert np.abs(out.double().cpu().numpy()[:, 0] - want).max() <= 8 * 4.4e-8 + 2.0 ** -24 + 2 * np.pi * 2.0 ** -28
    torch.testing.assert_close(out[8], q[8], rtol=0, atol=0)


@pytest.mark.parametrize("pairs,axes", [("half", 1), ("pair", 3)])
def test_rotated_float32_rows(pairs, axes):
    # off by 1.4 u (|a| + |b|) of cosine and sine, 1 u of each product and 1 u of their sum: 3.5 u (|a| + |b|)
    g = torch.Generator().manual_seed(axes)
    tokens, heads, d = 200, 3, 128
    q = torch.randn(tokens, heads, d, generator=g).cuda()
    pos = torch.randint(-9000, 9000, (axes, tokens), generator=g).cuda()
    inv = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float().cuda()
    axis = bytes(p % axes for p in range(d // 2)) if axes > 1 else None
    out = torch.empty_like(q)
    nrm.nrm_rope_fwd(q, None, pos, inv, out, None, axis=axis, pairs=pairs)
    x = q.double().cpu().numpy()
    want = ref.rotate(x, ref.angles(pos.cpu().numpy(), inv.cpu().numpy(), axis), pairs)
    lim = 3.5 * 2.0 ** -24 * ref.pair_size(x, d // 2, pairs)
    assert (np.abs(out.double().cpu().numpy() - want) <= lim).all()
