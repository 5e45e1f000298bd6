"""Sizes that the backward's workspace has no answer for are refused on the host."""
import pytest

import normalization_layernorm_rmsnorm_gb300 as nrm
from normalization_layernorm_rmsnorm_gb300 import _binding as B
from normalization_layernorm_rmsnorm_gb300 import build as nbuild

P = 1 << 20  # an aligned, non-null address that is never read: every call below is refused on the host


@pytest.mark.parametrize("tokens,d", [((1 << 32) + 1, 256), ((1 << 39) + 1, 2), ((1 << 40) // 255 + 1, 255)])
def test_backward_beyond_its_workspace_is_refused(tokens, d):
    nbuild.build()
    lib = nrm.load()
    # the workspace of such a call would be 0 bytes, which any workspace has
    assert nrm.nrm_workspace_bytes(nrm.NRM_OP_QK_NORM_BWD, tokens, d, nrm.NRM_F32) == 0
    rows = [B._Heads(i * P, 1, d, d) for i in range(1, 4)]
    status = lib.nrm_qk_norm_rope_bwd(rows[0], None, rows[1], None, None, None, P, None, None, rows[2], None, P, None,
                                      tokens, d, nrm.NRM_F32, P, 16, None)
    assert status == nrm.NRM_ERR_UNSUPPORTED and "2^40" in nrm.nrm_last_error_message()
