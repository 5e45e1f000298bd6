"""The handle of a cache holds the addresses of its tensors: they cannot be replaced under it."""
import copy

import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm

ATTRIBUTES = ("k_codes", "k_scales", "v_codes", "v_scales", "heads", "d", "slots", "held", "address")


@pytest.mark.parametrize("name", ATTRIBUTES)
def test_attributes_of_a_handle_cannot_be_set(name):
    # (a handle without its tensors, which need a GPU)
    cache = object.__new__(nrm.KvCache)
    with pytest.raises(AttributeError, match="kv_cache"):
        setattr(cache, name, None)
    with pytest.raises(AttributeError, match="deleted"):
        delattr(cache, name)


@pytest.mark.gpu
def test_a_handle_keeps_its_tensors():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    made = [torch.zeros(2, 4, 1, 64, dtype=torch.int8, device="cuda") for _ in range(2)]
    scales = [torch.zeros(2, 4, 1, 2, device="cuda") for _ in range(2)]
    cache = nrm.kv_cache(made[0], scales[0], made[1], scales[1])
    assert cache.k_codes is made[0] and cache.v_codes is made[1] and cache.held is made[0]
    assert cache.k_scales is scales[0] and cache.v_scales is scales[1]
    assert (cache.heads, cache.d, cache.slots) == (1, 64, 8)
    with pytest.raises(AttributeError):
        cache.k_codes = made[1]
    assert cache.k_codes is made[0] and copy.copy(cache) is cache
    x = torch.randn(8, 1, 64, device="cuda", dtype=torch.bfloat16)
    back, slots = torch.empty_like(x), torch.arange(8, device="cuda")
    del made, scales
    nrm.nrm_kv_cache_write(x, None, cache, slots)
    nrm.nrm_kv_cache_read(cache, slots, back, None)
    nrm.nrm_sync_status()
    # half a code's step, and bf16's rounding
    step = x.double().unflatten(-1, (2, 32)).abs().amax(-1, keepdim=True).expand(8, 1, 2, 32).flatten(-2) / 127
    assert ((back.double() - x.double()).abs() <= 0.5001 * step + 2.0 ** -8 * x.double().abs() * 1.01).all()
