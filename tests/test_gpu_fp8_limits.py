"""The e4m3 product at the limits it states (needs an MI355X): large terms that cancel beside small ones,
scales far from 1, either kernel for few rows."""
import numpy as np
import pytest
import torch

import selective_state_space_59_amd as ssm
from oracle import delta as R
from tests.recurrent_helpers import check, f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
IDS = dict(argvalues=[F32, BF], ids=["f32", "bf16"])
U = 2.0 ** -24
# the skinny kernel's range and the three tiles'
MATS = [(3, 130, 400), (65, 64, 256), (1237, 1331, 144), (4200, 4000, 400)]


def _call(xq, sx, wq, sw, dtype):
    dev = lambda t, d: torch.from_numpy(t).to(F32).to(d).to(DEV)  # noqa: E731
    e4m3 = torch.float8_e4m3fn
    return ssm.matmul_fp8(dev(xq, e4m3), dev(sx, F32), dev(wq, e4m3), dev(sw, F32), out_dtype=dtype)


def _tolerance(K, size, dtype):
    """A sum of K exact products in fp32 (twice a rounding for each, and the scales'); for a bf16 y the seven
    products of eight that the 8-bit instruction may cut at 2^-14 of the largest."""
    return (2 * (K + 4) * U + (7 * 2.0 ** -14 if dtype is BF else 0.0)) * size


@pytest.mark.parametrize("dtype", **IDS)
@pytest.mark.parametrize("M,N,K", MATS)
def test_large_terms_that_cancel(M, N, K, dtype):
    """Every eighth channel 448, with weights that cancel it in pairs, between values of 2^-6 to 4: what is
    left of the sum is up to 1e4 times smaller than its terms.  An fp32 result is right to 2^-24 of the terms,
    which still holds of each small one."""
    g = np.random.default_rng(M)
    xq, wq = (R.e4m3(np.exp2(g.uniform(-6, 2, s)) * g.choice([-1, 1], s)) for s in ((M, K), (N, K)))
    xq[:, ::8] = 448
    wq[:, ::16], wq[:, 8::16] = 448, -448
    kb = -(-K // 128)
    sx, sw = np.full((M, kb), 2.0 ** -3), np.full((-(-N // 128), kb), 2.0 ** -5)
    y = _call(xq, sx, wq, sw, dtype)
    want, size = R.matmul_blocks(xq, sx, wq, sw)
    check(y, want, _tolerance(K, size, dtype), "%dx%dx%d" % (M, N, K))


@pytest.mark.parametrize("dtype", **IDS)
@pytest.mark.parametrize("M,N,K", MATS)
@pytest.mark.parametrize("ex,ew", [(-100, 100), (100, -100), (-58, -60), (50, 44)])
def test_scales_far_from_1(ex, ew, M, N, K, dtype):
    """Products of scales from 2^-120 to 2^96, of factors that are larger and smaller."""
    g = np.random.default_rng(N)
    xq, wq = (R.e4m3(np.clip(100 * g.standard_normal(s), -448, 448)) for s in ((M, K), (N, K)))
    kb = -(-K // 128)
    scale = lambda e, n: f64(torch.from_numpy(np.exp2(e + g.uniform(-1, 1, (n, kb)))).float())  # noqa: E731
    sx, sw = scale(ex, M), scale(ew, -(-N // 128))
    y = _call(xq, sx, wq, sw, dtype)
    want, size = R.matmul_blocks(xq, sx, wq, sw)
    assert 1e-30 < np.abs(want).max() < 1e36
    check(y, want, _tolerance(K, size, dtype), "%dx%dx%d" % (M, N, K))


@pytest.mark.parametrize("dtype", **IDS)
@pytest.mark.parametrize("M,N,K", [(32, 8192, 144), (32, 8193, 144), (33, 4096, 272), (33, 4097, 272), (64, 4096, 144),
                                   (64, 6000, 144)])
def test_few_rows_of_either_kernel(M, N, K, dtype):
    """On both sides of where tiles take over from the skinny kernel."""
    g = np.random.default_rng(N + M)
    xq, wq = (R.e4m3(np.clip(100 * g.standard_normal(s), -448, 448)) for s in ((M, K), (N, K)))
    kb = -(-K // 128)
    sx, sw = (f64(torch.from_numpy(np.exp(g.standard_normal((n, kb)))).float()) for n in (M, -(-N // 128)))
    want, size = R.matmul_blocks(xq, sx, wq, sw)
    check(_call(xq, sx, wq, sw, dtype), want, _tolerance(K, size, dtype), "%dx%dx%d" % (M, N, K))
