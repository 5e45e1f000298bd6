"""The rotation's bits depend on a row, its position and the frequencies alone: not on alignment, strides,
the number of tokens or whether it runs in place, in a serving step or by itself."""
import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
from test_heads import CODES, Data, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    nrm.load()


def moved(x, offset, apart):
    """x's values `offset` elements into a buffer, `apart` elements between a token's rows and the next's."""
    tokens, heads, d = x.shape
    ts = heads * d + apart
    b = torch.zeros(tokens * ts + offset + 16, dtype=x.dtype, device="cuda")
    return b.as_strided((tokens, heads, d), (ts, d, 1), offset).copy_(x)


@pytest.mark.parametrize("pairs,axes", [("half", 1), ("pair", 2)])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 32), (256, 192)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rotation_does_not_depend_on_the_layout(dtype, d, rot, pairs, axes):
    c = Data(dtype, 60, 3, 2, d, rot, axes)
    how = dict(axis=c.axis, pairs=pairs)
    want = [torch.empty_like(t) for t in (c.q, c.k, c.q, c.k)]
    nrm.nrm_rope_fwd(c.q, c.k, c.pos, c.inv, *want[:2], **how)
    nrm.nrm_rope_bwd(c.dqo, c.dko, c.pos, c.inv, *want[2:], **how)
    for offset, apart in ((1, 0), (2, 0), (4, 0), (0, 1), (0, 2), (0, 4), (3, 7)):
        q, k, dq, dk = (moved(t, offset, apart) for t in (c.q, c.k, c.dqo, c.dko))
        got = [moved(torch.zeros_like(t), offset, apart) for t in (c.q, c.k, c.q, c.k)]
        nrm.nrm_rope_fwd(q, k, c.pos, c.inv, *got[:2], **how)
        nrm.nrm_rope_bwd(dq, dk, c.pos, c.inv, *got[2:], **how)
        nrm.nrm_rope_fwd(q, k, c.pos, c.inv, q, k, **how)  # in place
        for a, b in zip([*got, q, k], [*want, *want[:2]]):
            assert same(a, b), (offset, apart)
        # one token by itself
        one = torch.empty_like(c.q[7:8])
        nrm.nrm_rope_fwd(moved(c.q[7:8], offset, apart), None, c.pos[:, 7:8].contiguous(), c.inv, one, None, **how)
        assert same(one, want[0][7:8]), (offset, apart)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group", [2, 4, 8, 128])
def test_a_rotating_step_equals_its_parts_whatever_the_cache_allows(dtype, group):
    # the cache's groups and strides decide how wide the step's accesses are
    c = Data(dtype, 40, 4, 2, 128, 128)
    slots = torch.randperm(48, device="cuda")[:40]
    qo, ko, q2, k2 = (torch.empty_like(t) for t in (c.q, c.k, c.q, c.k))
    nrm.nrm_rope_fwd(c.q, c.k, c.pos, c.inv, qo, ko)
    for extra in (0, 1, 2, 4):  # bytes between the cache's rows
        def cache():
            codes = [torch.zeros(3, 16, 2, 128 + extra, dtype=torch.uint8, device="cuda")[..., :128].view(CODES["int8"])
                     for _ in range(2)]
            scales = [torch.zeros(3, 16, 2, 128 // group, device="cuda") for _ in range(2)]
            return nrm.kv_cache(codes[0], scales[0], codes[1], scales[1])

        one, two = cache(), cache()
        nrm.nrm_kv_cache_write(ko, c.v, one, slots)
        nrm.nrm_qk_norm_rope_cache(c.q, c.k, c.v, None, None, c.pos, c.inv, q2, k2, two, slots, 1e-6, norm=False)
        nrm.nrm_sync_status()
        assert same(q2, qo) and same(k2, ko)
        for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
            assert same(getattr(one, n), getattr(two, n)), (n, extra)
