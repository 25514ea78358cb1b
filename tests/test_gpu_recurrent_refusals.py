"""Arguments that the recurrence and the norms have to turn down (needs an MI355X)."""
import pytest
import torch

import selective_state_space_59_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_a_fraction_of_a_group():
    x, w = torch.randn(3, 48, device=DEV), torch.ones(48, device=DEV)
    want = ssm.gated_rmsnorm_fwd(x, x, w, groups=2)
    assert torch.equal(ssm.gated_rmsnorm_fwd(x, x, w, groups=2.0), want)
    for call in (lambda g: ssm.gated_rmsnorm_fwd(x, x, w, groups=g), lambda g: ssm.gated_rmsnorm(x, x, w, groups=g),
                 lambda g: ssm.gated_rmsnorm_bwd(x, x, w, x, groups=g)):
        with pytest.raises(ValueError, match="groups"):
            call(2.5)
