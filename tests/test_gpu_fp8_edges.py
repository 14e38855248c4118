"""The 8-bit projection path at its edges: results beyond float32, sums of one sign.

Sums of one sign.  The tensor core adds 32 products a step and cuts its sum off
towards zero, by one unit in the last place (2^-23 of the sum so far) at most.  Where
all products have one sign nothing cancels: the cuts of K columns add up to
K/32 2^-23 of the result at most, and as the sum grows evenly to half of that.
"""
import numpy as np
import pytest
import torch

import oracle
from parity import f64
from test_gpu_fp8 import D_NORM, bits, check_norm, exps, normal, proj_inputs, values
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


@pytest.mark.parametrize("T,d,dtype,residual", [
    (40000, 48, torch.bfloat16, False), (20000, 128, torch.bfloat16, True),   # rows of part of a warp
    (20000, 128, torch.float32, False), (12000, 256, torch.float32, True),
    (6000, 512, torch.bfloat16, True), (6000, 528, torch.bfloat16, False), (4000, 1040, torch.float32, True),
    (15000, 4096, torch.bfloat16, True), (15000, 2048, torch.float32, True),  # the short walks
    (15000, 4096, torch.bfloat16, False),
    (400, 16384, torch.float32, True), (400, 16384, torch.float32, False),    # no loads ahead
    (400, 32768, torch.bfloat16, True), (400, 32768, torch.float32, True),
])
def test_rmsnorm_of_more_rows_than_run_at_once(T, d, dtype, residual):
    """Blocks that walk several rows: every row equals, bit for bit, the same row in a
    batch so small that each block takes one, and sampled rows are right."""
    x = normal((T, d), dtype, T + d)
    res = normal((T, d), dtype, T + d + 1, 3.0) if residual else None
    gain = 1 + 0.3 * normal((d,), torch.float32, 2)
    whole = csa.rmsnorm_fp8(x, res, gain)
    piece = 100 if d >= 512 else 1000
    for a in range(0, T, piece):
        r = slice(a, min(T, a + piece))
        part = csa.rmsnorm_fp8(x[r], None if res is None else res[r], gain)
        for p, q in zip(part, whole):
            assert torch.equal(bits(p), bits(q[r])), a
    rows = [0, 1, T // 2, T - 2, T - 1]
    check_norm(x[rows], None if res is None else res[rows], gain, 1e-6, whole[0][rows],
               bits(whole[1])[rows])
    if residual:
        assert torch.equal(whole[2], (x.float() + res.float()).to(dtype))


# ---- fp8_matmul ----------------------------------------------------------------------

def one_signed(M, N, K, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((M, K), generator=gen, device=DEV).abs_()
    out = csa.fp8_quantize(x)
    del x
    return (*out, *csa.fp8_quantize(torch.randn((N, K), generator=gen, device=DEV).abs_(), 128))


def exact_product(xc, xs, wc, ws, step=8192):
    """x w^T in float64 on the device, `step` columns (a multiple of 128) at a time."""
    K, y = xc.shape[1], 0.0
    for k in range(0, K, step):
        e = min(K, k + step)
        x, w = (values(c.view(torch.uint8)[:, k:e].contiguous().view(torch.float8_e4m3fn),
                       s.view(torch.uint8)[:, k // 128:-(-e // 128)], rows)
                for c, s, rows in ((xc, xs, 1), (wc, ws, 128)))
        y = y + x @ w.t()
    return y


@pytest.mark.parametrize("M,N", [(1, 256), (40, 300), (2048, 1024)])
def test_matmul_longest_bf16_sum_of_one_sign(M, N):
    """A bf16 result's one sum at the longest K: the cut is an eighth of the rounding."""
    K = 1 << 17
    ops = one_signed(M, N, K, M)
    ref = exact_product(*ops)
    d = (csa.fp8_matmul(*ops).double() - ref).abs()
    assert bool((d <= (2.0 ** -8 * (1 + 2.0 ** -11) + K / 32 * 2.0 ** -23) * ref).all())


@pytest.mark.parametrize("M,N,K", [(5, 300, 1 << 20), (100, 10240, 1 << 16), (2048, 1536, 1 << 16)])
def test_matmul_float32_sums_of_one_sign_are_added_in_parts(M, N, K):
    """Each part's cut is at most half of 8192/32 2^-23 (and a sixteenth, as products are
    not all alike), a rounding for every part and share comes on top.  One sum of all
    columns that a share takes here (2^16 or 2^17) loses twice to four times that."""
    ops = one_signed(M, N, K, M)
    ref = exact_product(*ops)
    n0 = csa.csa_launch_count()
    y = csa.fp8_matmul(*ops, out_dtype=torch.float32).double()
    assert M > 128 or csa.csa_launch_count() - n0 > 1      # few rows: a launch a part
    rel = float(((y - ref).abs() / ref).max())
    assert rel <= 17 / 16 * 128 * 2.0 ** -23 + (K / 8192 + 8) * 2.0 ** -24, rel


@pytest.mark.parametrize("M,N,K", [
    (1, 640, 1 << 16), (3, 2000, 8192), (32, 300, 1 << 16), (100, 1000, 40000), (300, 520, 16384),
    (777, 1111, 1040), (2048, 1536, 16384), (2049, 2300, 8192),
])
def test_matmul_of_one_signed_integers_is_exact(M, N, K):
    """Whole numbers from 0 to 15, whose sums grow to 22 bits and stay below 2^24 at any
    K up to 2^16: a product that held fewer bits, or lost a column, would differ.  bf16
    results are the exact sums rounded once."""
    gen = torch.Generator(device=DEV).manual_seed(M + N + K)
    xc, xs = csa.fp8_quantize(torch.randint(0, 16, (M, K), generator=gen, device=DEV).float())
    wc, ws = csa.fp8_quantize(torch.randint(0, 16, (N, K), generator=gen, device=DEV).float(), 128)
    ref = exact_product(xc, xs, wc, ws)
    assert float(ref.max()) < 2 ** 24
    assert torch.equal(csa.fp8_matmul(xc, xs, wc, ws, out_dtype=torch.float32).double(), ref)
    assert torch.equal(csa.fp8_matmul(xc, xs, wc, ws), ref.float().bfloat16())


# ---- grouped_output_projection_fp8 ----------------------------------------------------

def test_projection_with_a_large_workspace_of_its_own_captured():
    """The call's own workspace, of which only the status word is zeroed, inside a graph
    that is replayed on other inputs."""
    x = proj_inputs(2000, 32, 512, 4, 256, 640, 1)      # 33 MB of codes
    y = torch.empty(2000, 640, dtype=torch.bfloat16, device=DEV)
    csa.grouped_output_projection_fp8(*x, y=y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa.grouped_output_projection_fp8(*x, y=y)
    for seed in (2, 3):
        x[0].copy_(proj_inputs(2000, 32, 512, 4, 256, 640, seed)[0])
        graph.replay()
        ws = csa.workspace(csa.csa_workspace_bytes(csa.CSA_OP_OUT_PROJ_FP8, torch.bfloat16, 1,
                                                   2000, 32, 512, 1024))
        assert torch.equal(y, csa.grouped_output_projection_fp8(*x, ws=ws))


def integer_weights(rows, cols, gen, top):
    """FP8 weights that are whole numbers from -top to top (at most 15: E4M3 holds them)."""
    return csa.fp8_quantize(torch.randint(-top, top + 1, (rows, cols), generator=gen,
                                          device=DEV).float(), 128)


@pytest.mark.parametrize("T,H,c,g,dg", [
    (4100, 32, 128, 4, 384),     # many rows: a last tile of 4 rows, half a tile past d_g
    (4100, 32, 128, 4, 640), (3100, 64, 256, 4, 128), (2048, 32, 128, 8, 1024),
    (300, 32, 128, 4, 384), (33, 8, 256, 2, 256), (1, 8, 256, 2, 128),   # few rows
])
def test_projection_intermediate_is_exact_on_integers(T, H, c, g, dg):
    """Whole numbers up to 15 and 7 in o and w_group: the grouped product's sums (below 2^24)
    are exact, and so are their codes; w_out is the unit matrix, whose product is the
    intermediate itself, in bf16 without a rounding.  A row that holds an infinity, and
    one whose sums are beyond float32, are NaN and leave the others alone."""
    gen = torch.Generator(device=DEV).manual_seed(T + dg)
    kg, gd = H // g * c, g * dg
    o = torch.randint(-15, 16, (T, H, c), generator=gen, device=DEV).bfloat16()
    wg, wgs = integer_weights(gd, kg, gen, 7)
    wo, wos = csa.fp8_quantize(torch.eye(gd, device=DEV), 128)
    bad = [T // 2, T - 1] if T > 2 else []
    if bad:
        o[bad[0], H // 2, 3] = float("inf")
        # codes and weights are finite, their sum is not: 2^127 a column, of the sign of
        # the first weight row's
        o[bad[1], :H // g] = torch.copysign(torch.tensor(2.0 ** 127, device=DEV),
                                            wg[0].float()).view(H // g, c).bfloat16()
    y = csa.grouped_output_projection_fp8(o, wg.view(g, dg, kg),
                                          wgs.view(g, dg // 128, kg // 128), wo, wos)
    assert bool(torch.isnan(y[bad]).all())
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[bad] = False
    w = values(wg, wgs, 128).view(g, dg, kg)
    v = torch.einsum("tgk,gnk->tgn", o[keep].double().view(-1, g, kg), w).reshape(-1, gd)
    assert float(v.abs().max()) < 2 ** 24
    assert np.array_equal(f64(y[keep]), oracle.fp8_values(*oracle.fp8_quantize(f64(v))))


@pytest.mark.parametrize("T", [5, 700, 3000])
def test_projection_repeats_itself(T):
    x = proj_inputs(T, 32, 128, 4, 512, 520, T)
    y = csa.grouped_output_projection_fp8(*x)
    for _ in range(3):
        assert torch.equal(csa.grouped_output_projection_fp8(*x), y)
