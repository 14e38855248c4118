"""The 8-bit projection path at its edges: results beyond float32."""
import numpy as np
import pytest
import torch

import oracle
from parity import f64
from test_gpu_fp8 import D_NORM, exps
import long_context_attention_csa_b200 as csa

pytestmark = pytest.mark.gpu

DEV = "cuda"


# ---- rmsnorm_fp8 ------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [48, 256, 528, 4096, 20480])
@pytest.mark.parametrize("wide", [False, True])
def test_rmsnorm_results_beyond_float32_are_nan(d, wide, dtype):
    """h gain is finite and y is not: those elements are NaN codes and leave the
    block's scale to the others.  h is 1/64, every fourth 3/64, so 1/rms is about
    36.9 and with a gain of 2e38 every fourth y is 3.46e38 (1.7% beyond the largest
    float32, far more than the kernel's relative error 2^-18), the others a third."""
    x = torch.full((5, d), 1 / 64, dtype=dtype, device=DEV)
    x[:, ::4] *= 3
    x[1] *= -1
    gain = torch.ones(d, device=DEV)
    gain[:d if wide else 40] = 2e38        # everywhere, or in a part of the first block
    codes, scales = csa.rmsnorm_fp8(x, gain=gain)
    _, y = oracle.rmsnorm_residual(f64(x), None, f64(gain), 1e-6)
    top = float(np.finfo(np.float32).max)
    over = np.abs(y) > top
    assert over.any() and (np.abs(y[over]) > 1.01 * top).all()
    y[over] = np.nan
    e = oracle.fp8_exponents(y)
    assert np.array_equal(exps(scales), e)
    got = f64(codes.float())
    assert np.array_equal(np.isnan(got), over)
    r = np.abs(np.ldexp(y, -oracle._fp8_spread(e, 1, y.shape)))[~over]
    half = np.ldexp(1.0, np.maximum(np.frexp(r * (1 + D_NORM))[1] - 1, -6) - 4)
    assert (np.abs(np.abs(got[~over]) - r) <= half + D_NORM * r).all()
