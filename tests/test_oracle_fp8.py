"""Pins for the oracle's 8-bit projection path: the block scale's definition,
the rounding against the E4M3 encoder that the indexer's pins cover and
against torch's conversion, the norm's closed forms and the projection's
limits."""
import numpy as np
import pytest
import torch

import oracle


def test_scale_is_the_smallest_power_of_two_that_holds_the_block():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((37, 300)) * np.exp2(rng.integers(-40, 40, (37, 1)))
    for rows in (1, 128):
        e = oracle.fp8_exponents(x, rows)
        assert e.shape == (-(-37 // rows), 3)
        for i in range(e.shape[0]):
            for j in range(3):
                a = np.abs(x[i * rows:(i + 1) * rows, 128 * j:128 * j + 128]).max()
                assert a <= 448 * 2.0 ** e[i, j] and a > 448 * 2.0 ** (e[i, j] - 1)


@pytest.mark.parametrize("amax,e", [(448.0, 0), (449.0, 1), (447.0, 0), (224.0, -1), (1.0, -8),
                                    (0.0, -127), (2.0 ** -149, -127), (3.4e38, 120)])
def test_scale_closed_forms(amax, e):
    x = np.zeros((1, 128))
    x[0, 77] = -amax
    assert oracle.fp8_exponents(x)[0, 0] == e


def test_nonfinite_elements_are_nan_codes_and_leave_the_scale():
    x = np.ones((1, 256))
    x[0, 3], x[0, 4], x[0, 5] = np.nan, np.inf, -np.inf
    c, e = oracle.fp8_quantize(x)
    assert np.isnan(c[0, 3:6]).all() and (e == -8).all()
    assert np.isfinite(np.delete(c[0], [3, 4, 5])).all()


def test_rounding_equals_the_encoder_and_torch():
    rng = np.random.default_rng(1)
    r = np.concatenate([rng.uniform(-448, 448, 2000), rng.standard_normal(2000) * 0.02,
                        [oracle.e4m3_value(c) for c in range(0x7F)],
                        [(oracle.e4m3_value(c) + oracle.e4m3_value(c + 1)) / 2
                         for c in range(0x7E)]])
    got = oracle.e4m3_round(r)
    want = np.array([oracle.e4m3_value(oracle.e4m3_encode(v)) for v in r])
    assert np.array_equal(got, want)
    t = torch.from_numpy(r).to(torch.float32).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(oracle.e4m3_round(r.astype(np.float32)), t)


def test_values_round_trip_representable_blocks():
    rng = np.random.default_rng(2)
    c = np.array([oracle.e4m3_value(int(v)) for v in rng.integers(0, 0x7E, 5 * 128)]).reshape(5, 128)
    c[:, 0] = 448.0
    x = np.ldexp(c, rng.integers(-20, 20, (5, 1)))
    assert np.array_equal(oracle.fp8_values(*oracle.fp8_quantize(x)), x)


def test_norm_closed_forms():
    h, y = oracle.rmsnorm_residual(np.full((2, 8), 3.0), np.full((2, 8), 1.0), eps=0.0)
    assert (h == 4.0).all() and np.allclose(y, 1.0, rtol=1e-15)
    x = np.random.default_rng(3).standard_normal((4, 48))
    _, y = oracle.rmsnorm_residual(x, eps=1e-6)
    assert np.allclose(y, np.stack([oracle.rmsnorm(r) for r in x]), rtol=1e-12)
    _, g = oracle.rmsnorm_residual(x, gain=np.arange(48.0))
    assert np.allclose(g, y * np.arange(48.0), rtol=1e-12)


def test_projection_of_representable_rows_is_the_plain_projection():
    """Rows and intermediates that E4M3 holds exactly: the quantizations change nothing."""
    o = np.zeros((3, 4, 64))
    o[:, :, :] = np.array([1.0, -2.0, 0.5])[:, None, None]
    w_group = np.zeros((2, 128, 128))
    w_group[:, np.arange(128), np.arange(128)] = 1.0
    w_out = np.random.default_rng(4).standard_normal((5, 256))
    assert np.allclose(oracle.grouped_output_projection_fp8(o, w_group, w_out),
                       oracle.grouped_output_projection(o, w_group, w_out), rtol=1e-12)
