"""Workspace sizes of the add + norm backward (host only): what its options need, as the header says."""
import ctypes

import pytest

from selective_state_space_59_amd import ssm

ADDRESS = 0x7F0000000000


@pytest.mark.parametrize("io", [ssm.SSM_F32, ssm.SSM_BF16])
@pytest.mark.parametrize("rows,dim", [(1, 8), (5000, 64), (70000, 64), (3000, 768), (3000, 1280), (9, 4100), (300, 9000)])
def test_add_norm_backward_is_sized_by_its_options(rows, dim, io):
    """One column sum (w), two with a scale, three with a post norm: each takes the same rows of partial
    sums and the same scratch, up to the 256 bytes each part is rounded up to."""
    def size(**kw):
        a = ssm.AddNormBwdArgs(rows=rows, dim=dim, io_dtype=io, res_dtype=io, eps=1e-5, **kw)
        return ssm.lib().ssm_add_rmsnorm_bwd_workspace_size(ctypes.byref(a))

    plain, scale, post = size(), size(scale=ADDRESS), size(post_w=ADDRESS)
    assert post == size(scale=ADDRESS, post_w=ADDRESS)
    assert 0 < plain <= scale <= post
    assert abs(scale - 2 * plain) <= 4 * 256 and abs(post - 3 * plain) <= 6 * 256
