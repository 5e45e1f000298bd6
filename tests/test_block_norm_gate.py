"""A gate without rows is no gate of 1."""
import pytest
import torch

import normalization_layernorm_rmsnorm_gb300 as nrm
from test_served_host import _rows, lib  # noqa: F401


def test_a_gate_without_rows_is_refused(lib):  # noqa: F811
    empty = torch.zeros(0, 16)
    with pytest.raises(ValueError, match="gate has no rows"):
        nrm.nrm_block_norm_fwd(**_rows(gate=empty))
    t, r = torch.zeros(6, 16), torch.zeros(6)
    a = dict(dh=t, dy=t, f=t, y=t, gate=empty, w_post=None, w_pre=None, rstd_post=r, rstd_pre=r, dx=t, df=t, dgate=empty,
             dw_post=None, dw_pre=None, workspace=None, alpha=1.0)
    with pytest.raises(ValueError, match="gate has no rows"):
        nrm.nrm_block_norm_bwd(**a)
    # without rows of x it is one
    e = torch.zeros(0, 16)
    with pytest.raises(ValueError, match="current CUDA device"):
        nrm.nrm_block_norm_fwd(e, e, empty, None, None, e, e, None, None, 1.0, 1e-6)
