"""The fused norms on both sides of every width at which they take another launch shape, with more
rows than a launch walks over at once, against the fp64 definitions (needs an MI355X)."""
import pytest
import torch

from tests import test_gpu_norms as norms

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("io", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("gate_first", [True, False], ids=["gate_first", "norm_first"])
@pytest.mark.parametrize("rows,D,groups", [
    (2100, 256, 1), (37, 257, 1), (2100, 512, 1), (5, 520, 1), (11, 1026, 2), (900, 2052, 4), (2500, 768, 1),
    (2300, 769, 1), (700, 1000, 2), (9, 1023, 1), (1100, 1536, 3), (1100, 2307, 3), (2100, 1024, 1), (600, 2050, 2),
    (4300, 65, 1), (1100, 640, 5)])
def test_gated_rmsnorm(rows, D, groups, gate_first, io):
    """Waves of one and two groups a lane, whose column sums meet in a workgroup, beside half waves,
    quarter waves and workgroups; one to five groups."""
    norms.test_gated_rmsnorm(rows, D, groups, gate_first, io)


@pytest.mark.parametrize("io,res", norms.TYPES, ids=["f32_f32", "bf16_bf16", "bf16_f32", "f32_bf16"])
@pytest.mark.parametrize("rows,D", [(4300, 65), (2100, 257), (2100, 512), (2100, 513), (2300, 769), (2100, 1024),
                                    (1100, 1025)])
def test_add_rmsnorm(rows, D, io, res):
    norms.test_add_rmsnorm(rows, D, io, res)
