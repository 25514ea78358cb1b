"""The gated delta rule at its largest value width (needs an MI355X)."""
import pytest
import torch

from tests.delta_helpers import delta_case
from tests.test_gpu_gated_delta import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 70, 1, 2, 128, 1024), (1, 130, 2, 2, 8, 1024), (3, 66, 1, 4, 72, 1016)],
                         ids=lambda s: "x".join(map(str, s)))
def test_values_of_up_to_1024_channels(shape, dtype):
    """64 slices of a chain, sums over them, 32 passes of the gradients; a last chunk that is not whole."""
    for ck in (True, False):
        _check(delta_case(*shape, dtype, seed=sum(shape), doc=40, beta=2.0), "%s ck=%d" % (shape, ck), checkpoints=ck)
