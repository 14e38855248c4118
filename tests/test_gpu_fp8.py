"""GPU parity of the 8-bit projection path (rmsnorm_fp8, fp8_quantize,
fp8_matmul, grouped_output_projection_fp8) against the float64 oracle.

Tolerances.  fp8_quantize: bit-exact (the scaling by a power of two is exact
and there is one rounding).  rmsnorm_fp8: the float32 value before the codes is
off by a relative D = 2^-18 at most: the row's sum of squares adds up to 64
products a thread, 5 shuffle steps and 16 warps (85 roundings, halved by the
square root), h, the reciprocal root and two products round at most 7 times
more: 50 x 2^-24 < 2^-18; then E4M3's half step of the exact value.  fp8_matmul:
products of two codes are exact in float32, and every one of the K additions
loses at most one unit in the last place (2^-23, a truncating adder) of a
partial sum bounded by S = sum |x||w|: K 2^-23 S elementwise.  Over a whole
matrix partial sums are of the size of the result and the tensor core adds 32
products at a time: K / 32 + 32 losses of 2^-23 bound the relative 2-norm.  The
output's own rounding adds half a step (bf16 2^-8, float32 2^-24 relative).
"""
import numpy as np
import pytest
import torch

import oracle
from parity import f64
import long_context_attention_csa_b200 as csa
from long_context_attention_csa_b200 import workloads as wl

pytestmark = pytest.mark.gpu

DEV = "cuda"
D_NORM = 2.0 ** -18
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def exps(scales):
    return scales.view(torch.uint8).cpu().numpy().astype(np.int64) - 127


def normal(shape, dtype, seed, scale=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)


def same_codes(codes, want):
    """E4M3 values equal, NaN where NaN."""
    return np.array_equal(f64(codes.float()), want, equal_nan=True)


# ---- fp8_quantize ---------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,d", [(1, 16), (1, 4096), (3, 144), (127, 128), (129, 272),
                                    (300, 1040), (1000, 32)])
def test_quantize_is_exact(rows, d, block_rows, dtype):
    x = normal((rows, d), dtype, rows + d)
    x *= torch.exp2(torch.randint(-30, 30, (rows, 1), device=DEV).float()).to(dtype)
    codes, scales = csa.fp8_quantize(x, block_rows)
    want, e = oracle.fp8_quantize(f64(x), block_rows)
    assert codes.dtype == torch.float8_e4m3fn and scales.dtype == torch.float8_e8m0fnu
    assert np.array_equal(exps(scales), e)
    assert same_codes(codes, want)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_extremes(block_rows):
    x = torch.zeros(130, 400, device=DEV)
    x[0, :128] = torch.linspace(-448, 448, 128)
    x[1, 128:256] = 3.3e38
    x[2, 256:] = 2.0 ** -149
    x[3, 0] = float("nan")
    x[4, 1], x[4, 2], x[4, 3] = float("inf"), float("-inf"), 5.0
    x[5, 128:256] = float("nan")
    x[6, 128:256] = float("inf")
    x[7, 256:] = -0.0
    x[129] = 448.0 * (1 + 2.0 ** -20)
    for dtype in (torch.float32, torch.bfloat16):
        codes, scales = csa.fp8_quantize(x.to(dtype), block_rows)
        want, e = oracle.fp8_quantize(f64(x.to(dtype)), block_rows)
        assert np.array_equal(exps(scales), e)
        assert same_codes(codes, want)


def test_quantize_row_stride_and_shapes():
    wide = normal((70, 512), torch.bfloat16, 5)
    part = wide[:, 128:384]
    c0, s0 = csa.fp8_quantize(part)
    c1, s1 = csa.fp8_quantize(part.contiguous())
    assert torch.equal(c0.view(torch.uint8), c1.view(torch.uint8))
    assert torch.equal(s0.view(torch.uint8), s1.view(torch.uint8))
    c2, s2 = csa.fp8_quantize(wide.view(7, 10, 512))
    assert c2.shape == (7, 10, 512) and s2.shape == (7, 10, 4)
    c3, s3 = csa.fp8_quantize(wide[:0])
    assert c3.shape == (0, 512) and s3.shape == (0, 4)


def bits(t):
    return t.view(torch.uint8) if t.element_size() == 1 else t


@pytest.mark.parametrize("dtype,shift", [(torch.bfloat16, 8), (torch.float32, 4)])
def test_rows_on_16_byte_boundaries(dtype, shift):
    """Rows that start 16 bytes off a 32-byte boundary, in every operand."""
    def off(t):   # the same values, 16 bytes into a wider buffer
        wide = torch.zeros(t.shape[0], t.shape[1] + 2 * shift, dtype=t.dtype, device=DEV)
        wide[:, shift:-shift] = t
        return wide[:, shift:-shift]

    x, r = normal((150, 528), dtype, 1), normal((150, 528), dtype, 2)
    xo, ro = off(x), off(r)
    assert xo.data_ptr() % 32 == 16
    for br in (1, 128):
        for a, b in zip(csa.fp8_quantize(xo, br), csa.fp8_quantize(x, br)):
            assert torch.equal(bits(a), bits(b))
    for a, b in zip(csa.rmsnorm_fp8(xo, ro, sum_out=ro), csa.rmsnorm_fp8(x, r)):
        assert torch.equal(bits(a), bits(b))


def test_quantize_past_2_31_elements():
    """Offsets beyond 32 bits, in the input and in the codes."""
    rows, d = 66000, 32768
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device=DEV)
    x[-1] = normal((d,), torch.bfloat16, 1)
    codes, scales = csa.fp8_quantize(x)
    want, e = oracle.fp8_quantize(f64(x[-1:]))
    assert np.array_equal(exps(scales[-1:]), e) and same_codes(codes[-1:], want)
    assert int(scales[-2].view(torch.uint8).max()) == 0
    del codes, scales
    codes, scales = csa.fp8_quantize(x, 128)
    want, e = oracle.fp8_quantize(f64(x[rows // 128 * 128:]), 128)
    assert np.array_equal(exps(scales[-1:]), e) and same_codes(codes[rows // 128 * 128:], want)


# ---- rmsnorm_fp8 ------------------------------------------------------------------

def check_norm(x, res, gain, eps, codes, scales, what=""):
    _, y = oracle.rmsnorm_residual(f64(x), None if res is None else f64(res),
                                   None if gain is None else f64(gain), eps)
    e = exps(scales)
    nb = e.shape[1]
    full = np.zeros((y.shape[0], nb * 128))
    full[:, :y.shape[1]] = np.abs(y)
    amax = full.reshape(-1, nb, 128).max(axis=2)
    assert (amax * (1 - D_NORM) <= np.ldexp(448.0, e)).all(), what
    assert ((amax * (1 + D_NORM) > np.ldexp(448.0, e - 1)) | (e == -127)).all(), what
    r = np.ldexp(y, -oracle._fp8_spread(e, 1, y.shape))
    a = np.abs(r)
    half = np.ldexp(1.0, np.maximum(np.frexp(np.maximum(a * (1 + D_NORM), 2.0 ** -40))[1] - 1, -6) - 4)
    got = f64(codes.float())
    # at the very top 448 holds what the smaller value's rounding sends there
    assert (np.abs(got - r) <= half + D_NORM * a).all(), (
        what, float((np.abs(got - r) - half - D_NORM * a).max()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(1, 16), (1, 4096), (5, 80), (33, 512), (300, 528), (7, 1040),
                                 (2, 2064), (129, 4096), (3, 16384), (2, 32768)])
@pytest.mark.parametrize("residual,gain", [(True, True), (False, False)])
def test_rmsnorm(T, d, residual, gain, dtype):
    x = normal((T, d), dtype, T + d)
    res = normal((T, d), dtype, T + d + 1, 3.0) if residual else None
    g = 1 + 0.3 * normal((d,), torch.float32, 2) if gain else None
    out = csa.rmsnorm_fp8(x, res, g)
    check_norm(x, res, g, 1e-6, out[0], out[1])
    if residual:
        assert torch.equal(out[2], (x.float() + res.float()).to(dtype))
    else:
        assert len(out) == 2


def test_rmsnorm_extremes():
    """Squares beyond float32, rows of zeros, tiny rows, an infinity, a NaN."""
    x = normal((8, 640), torch.float32, 3)
    x[1] *= 1e25
    x[2] = 0.0
    x[3] *= 1e-30
    x[4, 7] = float("inf")
    x[5, 9] = float("nan")
    x[6, 0] = 1e38
    codes, scales = csa.rmsnorm_fp8(x)
    fine = [0, 1, 2, 3, 6, 7]
    check_norm(x[fine], None, None, 1e-6, codes[fine], scales[fine])
    c = f64(codes.float())
    assert np.isnan(c[4, 7]) and (np.delete(c[4], 7) == 0).all()
    assert np.isnan(c[5]).all()
    assert (c[2] == 0).all() and (exps(scales)[2] == -127).all()


@pytest.mark.parametrize("d", [48, 640, 4096, 20480])
def test_rmsnorm_of_rows_at_the_ends_of_float32(d):
    """Squares that float32 does not hold, where eps does not hide them either."""
    for eps in (0.0, float(np.float32(2.0 ** -133))):
        x = normal((6, d), torch.float32, d)
        for i, s in enumerate((2.0 ** -66, 2.0 ** -80, 2.0 ** -140, 2.0 ** 100, 1.0, 2.0 ** -50)):
            x[i] *= s
        g = 1 + 0.3 * normal((d,), torch.float32, 2)
        for gain in (None, g):
            codes, scales = csa.rmsnorm_fp8(x, None, gain, eps)
            check_norm(x, None, gain, eps, codes, scales, eps)
    x = normal((3, d), torch.float32, 1, 1e25)
    codes, scales = csa.rmsnorm_fp8(x, eps=1e38)
    check_norm(x, None, None, float(np.float32(1e38)), codes, scales)


def test_rmsnorm_in_place_and_strided():
    x, r = normal((37, 512), torch.bfloat16, 8), normal((37, 512), torch.bfloat16, 9)
    want = csa.rmsnorm_fp8(x, r)
    wide = torch.zeros(37, 1024, dtype=torch.bfloat16, device=DEV)
    wide[:, 512:] = r
    into = wide[:, 512:]
    got = csa.rmsnorm_fp8(x, into, sum_out=into)       # the residual stream updated in place
    for a, b in zip(got, want):
        assert torch.equal(bits(a), bits(b))
    assert (wide[:, :512] == 0).all()
    x2 = x.clone()
    csa.rmsnorm_fp8(x2, r, sum_out=x2)
    assert torch.equal(x2, want[2])


def test_rmsnorm_rows_do_not_depend_on_the_batch():
    x, r = normal((700, 4096), torch.bfloat16, 4), normal((700, 4096), torch.bfloat16, 5)
    all_ = csa.rmsnorm_fp8(x, r)
    for t in (0, 311, 699):
        one = csa.rmsnorm_fp8(x[t:t + 1], r[t:t + 1])
        assert torch.equal(one[0].view(torch.uint8)[0], all_[0].view(torch.uint8)[t])
        assert torch.equal(one[1].view(torch.uint8)[0], all_[1].view(torch.uint8)[t])


# ---- fp8_matmul ----------------------------------------------------------------------

def operands(M, N, K, seed, integers=False):
    if integers:
        gen = torch.Generator(device=DEV).manual_seed(seed)
        x = torch.randint(-3, 4, (M, K), generator=gen, device=DEV).float()
        w = torch.randint(-3, 4, (N, K), generator=gen, device=DEV).float()
    else:
        x = normal((M, K), torch.float32, seed)
        x *= torch.exp2(torch.randint(-6, 6, (M, 1), device=DEV).float())
        w = normal((N, K), torch.float32, seed + 1, K ** -0.5)
    return (*csa.fp8_quantize(x), *csa.fp8_quantize(w, 128))


def values(codes, scales, rows):
    """Float64 values on the device."""
    e = scales.view(torch.uint8).double() - 127
    e = e.repeat_interleave(rows, 0).repeat_interleave(128, 1)[:codes.shape[0], :codes.shape[1]]
    return codes.double() * torch.exp2(e)


def check_matmul(y, xc, xs, wc, ws, what=""):
    K = xc.shape[1]
    x, w = values(xc, xs, 1), values(wc, ws, 128)
    ref, S = x @ w.t(), x.abs() @ w.abs().t()
    d = (y.double() - ref).abs()
    bound = K * 2.0 ** -23 * S + HALF[y.dtype] * ref.abs()
    assert bool((d <= bound).all()), (what, float((d / bound.clamp(min=1e-300)).max()))
    rel = float(d.norm() / ref.norm().clamp(min=1e-300))
    assert rel <= (K / 32 + 32) * 2.0 ** -23 + HALF[y.dtype], (what, rel)
    return rel


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 16), (1, 128, 128), (1, 8192, 4096), (2, 131, 144), (16, 256, 512), (17, 129, 528),
    (32, 1000, 4096), (33, 257, 640), (64, 520, 1024), (65, 512, 2064), (100, 300, 16384),
    (128, 256, 512), (129, 257, 1040), (200, 1111, 272), (257, 4096, 768), (513, 999, 1552),
    (1000, 1024, 4096), (2049, 2300, 1024), (2049, 4090, 2048), (1100, 4097, 2064),
    (700, 16384, 528), (4096, 4104, 1040),
])
def test_matmul(M, N, K, out):
    xc, xs, wc, ws = operands(M, N, K, M + N + K)
    y = csa.fp8_matmul(xc, xs, wc, ws, out_dtype=out)
    assert y.dtype == out and y.shape == (M, N)
    check_matmul(y, xc, xs, wc, ws)


@pytest.mark.parametrize("M,N,K", [(1, 640, 1024), (40, 130, 2048), (300, 520, 400),
                                   (1500, 1300, 256)])
def test_matmul_of_integers_is_exact(M, N, K):
    xc, xs, wc, ws = operands(M, N, K, 7, integers=True)
    y = csa.fp8_matmul(xc, xs, wc, ws, out_dtype=torch.float32)
    assert torch.equal(y.double(), values(xc, xs, 1) @ values(wc, ws, 128).t())


@pytest.mark.parametrize("M,N,K", [(2048, 1536, 16992), (2048, 1531, 16384), (2048, 1536, 24576),
                                   (700, 1000, 20000), (1700, 300, 24576), (40, 4000, 70000),
                                   (5, 1000, 65552), (100, 2000, 32784), (33, 300, 16400)])
def test_matmul_long_float32_sums_are_added_in_parts(M, N, K):
    """float32 results of a K beyond 8192 a share are the rounded sums of the parts."""
    xc, xs, wc, ws = operands(M, N, K, 12)
    y = csa.fp8_matmul(xc, xs, wc, ws, out_dtype=torch.float32)
    rel = check_matmul(y, xc, xs, wc, ws)
    # each part's loss is bounded as a product of its own length
    assert rel <= (min(K, 8192) / 32 + 32) * 2.0 ** -23
    wide = torch.full((M, N + 3), 5.0, device=DEV)
    csa.fp8_matmul(xc, xs, wc, ws, y=wide[:, 1:N + 1])      # rows that start anywhere
    assert torch.equal(wide[:, 1:N + 1], y)
    assert (wide[:, 0] == 5).all() and (wide[:, N + 1:] == 5).all()
    if M == 2048 and K % 8192 == 0:   # accumulators of 8192 columns, added in order
        cut = [(k, min(k + 8192, K)) for k in range(0, K, 8192)]
        part = [csa.fp8_matmul(*(f.view(torch.uint8)[:, k // n:e // n].contiguous()
                                 for f, n in ((xc, 1), (xs, 128), (wc, 1), (ws, 128))),
                               out_dtype=torch.float32) for k, e in cut]
        total = part[0]
        for p in part[1:]:
            total = total + p
        assert torch.equal(total, y)


def test_matmul_added_in_parts_replays():
    """A captured call whose result is added up in Y starts over at every replay."""
    xc, xs, wc, ws = operands(2048, 1536, 16384, 5)
    room = csa.workspace(256)
    want = csa.fp8_matmul(xc, xs, wc, ws, torch.float32, ws=room)
    y = torch.full_like(want, float("nan"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa.fp8_matmul(xc, xs, wc, ws, y=y, ws=room)
    for _ in range(3):
        graph.replay()
    assert torch.equal(y, want)


def test_matmul_of_slices_of_a_batch():
    """Rows from the middle of a batch: scales that start anywhere."""
    xc, xs, wc, ws = operands(900, 300, 1168, 9)
    for a, b in ((1, 2), (3, 40), (7, 300), (899, 900), (0, 900)):
        y = csa.fp8_matmul(xc[a:b], xs[a:b], wc, ws)
        check_matmul(y, xc[a:b], xs[a:b], wc, ws)


def test_matmul_into_an_aligned_slice_by_pairs():
    """The many-row kernel into column slices that start 16 and 32 bytes apart."""
    xc, xs, wc, ws = operands(2048, 2048, 2048, 5)
    want = csa.fp8_matmul(xc, xs, wc, ws)
    check_matmul(want, xc, xs, wc, ws)
    for at in (0, 8, 16):
        wide = torch.full((2050, 2048 + 48), 9.0, dtype=torch.bfloat16, device=DEV)
        csa.fp8_matmul(xc, xs, wc, ws, y=wide[:2048, at:at + 2048])
        assert torch.equal(wide[:2048, at:at + 2048], want)
        assert (wide[:2048, :at] == 9).all() and (wide[:2048, at + 2048:] == 9).all()
        assert (wide[2048:] == 9).all()


def test_matmul_into_a_slice_leaves_the_rest():
    """Two projections into one wide buffer, and rows and columns beside them untouched."""
    for M in (5, 70, 300):
        xc, xs, wc, ws = operands(M, 200, 512, M)
        wide = torch.full((M + 3, 517), 9.0, dtype=torch.bfloat16, device=DEV)
        csa.fp8_matmul(xc, xs, wc, ws, y=wide[:M, 3:203])
        csa.fp8_matmul(xc, xs, wc, ws, y=wide[:M, 203:403])
        want = csa.fp8_matmul(xc, xs, wc, ws)
        assert torch.equal(wide[:M, 3:203], want) and torch.equal(wide[:M, 203:403], want)
        assert (wide[:, :3] == 9).all() and (wide[:, 403:] == 9).all() and (wide[M:] == 9).all()


@pytest.mark.parametrize("M", [3, 400])
def test_matmul_extreme_scales_and_nan(M):
    """Blocks of zeros, far apart scales, NaN codes and a NaN scale stay in their rows."""
    xc, xs, wc, ws = operands(M, 150, 384, 11)
    xs = xs.view(torch.uint8).clone()
    xc = xc.view(torch.uint8).clone()
    ws = ws.view(torch.uint8).clone()
    xc[0, 128:256] = 0
    xs[0, 1] = 0                     # an empty block's scale
    xs[1] = torch.tensor([200, 60, 127], dtype=torch.uint8)
    xc[2, 5] = 0x7F                  # NaN
    y = csa.fp8_matmul(xc, xs, wc, ws, out_dtype=torch.float32)
    assert bool(torch.isnan(y[2]).all())
    keep = [r for r in range(M) if r != 2]
    check_matmul(y[keep], xc.view(torch.float8_e4m3fn)[keep], xs[keep],
                 wc, ws)
    xs[2, 0] = 255                   # NaN
    xc[2, 5] = 0
    y2 = csa.fp8_matmul(xc, xs, wc, ws, out_dtype=torch.float32)
    assert bool(torch.isnan(y2[2]).all()) and torch.equal(y2[keep], y[keep])


def test_matmul_rows_do_not_depend_on_their_neighbours():
    for M in (20, 600):
        xc, xs, wc, ws = operands(M, 384, 1024, 3)
        y = csa.fp8_matmul(xc, xs, wc, ws)
        xc2, xs2 = xc.view(torch.uint8).clone(), xs.view(torch.uint8).clone()
        xc2[:-1], xs2[:-1] = 0x41, 130
        y2 = csa.fp8_matmul(xc2, xs2, wc, ws)
        assert torch.equal(y[-1], y2[-1])


def test_matmul_output_past_2_31_elements():
    M, N, K = 140000, 16384, 64
    xc, xs, wc, ws = operands(M, N, K, 1)
    y = csa.fp8_matmul(xc, xs, wc, ws)
    rows = torch.tensor([0, 1, 65537, M // 2, M - 2, M - 1], device=DEV)
    check_matmul(y[rows], xc.view(torch.uint8)[rows].view(torch.float8_e4m3fn),
                 xs.view(torch.uint8)[rows], wc, ws)


def test_matmul_refuses_before_launching():
    xc, xs, wc, ws = operands(4, 8, 256, 0)
    u8 = torch.uint8
    bad = [
        lambda: csa.fp8_matmul(xc, xs[:2], wc, ws),
        lambda: csa.fp8_matmul(xc, xs, wc, xs),
        lambda: csa.fp8_matmul(xc.float(), xs, wc, ws),
        lambda: csa.fp8_matmul(xc.view(u8).t().contiguous().t(), xs, wc, ws),
        lambda: csa.fp8_matmul(xc, xs, wc[:, :128], ws),
        lambda: csa.fp8_matmul(xc, xs, wc, ws.cpu()),
        lambda: csa.fp8_matmul(xc, xs, wc, ws, out_dtype=torch.float16),
        lambda: csa.fp8_matmul(xc, xs, wc, ws, y=torch.empty(4, 9, device=DEV)),
        lambda: csa.fp8_matmul(xc, xs, wc, ws, ws=torch.zeros(16, dtype=u8, device=DEV)),
    ]
    n0 = csa.csa_launch_count()
    for call in bad:
        with pytest.raises(csa.CSAError):
            call()
    assert csa.csa_launch_count() == n0


# ---- grouped_output_projection_fp8 -----------------------------------------------------

def proj_inputs(T, H, c, g, dg, d, seed, dtype=torch.bfloat16):
    o = normal((T, H, c), dtype, seed)
    kg = H // g * c
    wg, wgs = csa.fp8_quantize(normal((g * dg, kg), torch.float32, seed + 1, kg ** -0.5), 128)
    wo, wos = csa.fp8_quantize(normal((d, g * dg), torch.float32, seed + 2, (g * dg) ** -0.5), 128)
    return o, wg.view(g, dg, kg), wgs.view(g, dg // 128, kg // 128), wo, wos


def check_proj(y, o, wg, wgs, wo, wos, what=""):
    """v's codes may fall to the other side of a rounding border where the
    float32 sums differ from the exact ones: by (K/32 + 32) 2^-23 of v's size
    in the 2-norm, a share 2^4 times that of the codes by one step (2^-3): the
    relative 2-norm of v is off by sqrt(2^4 r) 2^-3, and y's by as much."""
    g, dg, kg = wg.shape
    wgv = torch.stack([values(wg[j], wgs[j], 128) for j in range(g)])
    ref = oracle.grouped_output_projection_fp8(f64(o), f64(wgv), f64(values(wo, wos, 128)))
    got = f64(y)
    r = (kg / 32 + 32) * 2.0 ** -23
    rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert rel <= np.sqrt(16 * r) / 8 + 2.0 ** -8, (what, rel)
    return rel


@pytest.mark.parametrize("T,H,c,g,dg,d", [
    (1, 64, 512, 8, 1024, 4096), (5, 4, 64, 2, 128, 96), (32, 8, 128, 4, 256, 515),
    (130, 16, 64, 8, 128, 256), (300, 16, 512, 4, 384, 1001), (700, 8, 128, 1, 1024, 520),
])
def test_projection(T, H, c, g, dg, d):
    x = proj_inputs(T, H, c, g, dg, d, T)
    check_proj(csa.grouped_output_projection_fp8(*x), *x)


def test_projection_of_float32_rows():
    x = proj_inputs(70, 8, 64, 2, 128, 200, 1, torch.float32)
    check_proj(csa.grouped_output_projection_fp8(*x), *x)


def test_projection_with_a_workspace_on_a_16_byte_boundary():
    for T in (20, 3000):
        x = proj_inputs(T, 8, 256, 4, 256, 640, T)
        n = csa.csa_workspace_bytes(csa.CSA_OP_OUT_PROJ_FP8, torch.bfloat16, 1, T, 8, 256, 1024)
        ws = csa.workspace(n + 16)[16:]
        assert ws.data_ptr() % 32 == 16
        assert torch.equal(csa.grouped_output_projection_fp8(*x, ws=ws),
                           csa.grouped_output_projection_fp8(*x))
        assert csa.csa_check_status(ws) == (csa.CSA_OK, 0)


def test_projection_8k_sampled():
    """The 8192-row projection against the same rows' oracle."""
    x = proj_inputs(8192, 64, 512, 8, 1024, 4096, 2)
    y = csa.grouped_output_projection_fp8(*x)
    rows = [0, 1, 127, 128, 4095, 8190, 8191]
    check_proj(y[rows], x[0][rows], *x[1:])


# ---- streams, graphs, two calls at once ----------------------------------------------

def test_other_streams_and_captured_graphs():
    """Calls on a side stream, the same calls captured and replayed on new
    inputs, and two graphs that share one workspace replayed in turn."""
    x, r = normal((48, 1024), torch.bfloat16, 1), normal((48, 1024), torch.bfloat16, 2)
    wc, wsc = csa.fp8_quantize(normal((520, 1024), torch.float32, 3, 1 / 32), 128)
    o, wg, wgs, wo, wos = proj_inputs(48, 8, 128, 2, 256, 300, 4)
    ws = csa.workspace(csa.csa_workspace_bytes(csa.CSA_OP_OUT_PROJ_FP8, torch.bfloat16, 1, 48, 8,
                                               128, 512))

    def step():
        c, s, h = csa.rmsnorm_fp8(x, r)
        return csa.fp8_matmul(c, s, wc, wsc, ws=ws), h

    def project():
        return csa.grouped_output_projection_fp8(o, wg, wgs, wo, wos, ws=ws)

    want, want_p = step(), project()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, got_p = step(), project()
        g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(got_p, want_p)
    with torch.cuda.graph(g1, stream=side):
        out = step()
    with torch.cuda.graph(g2, stream=side):
        out_p = project()
    x.copy_(normal((48, 1024), torch.bfloat16, 21))
    o.copy_(normal((48, 8, 128), torch.bfloat16, 22))
    for _ in range(3):
        g1.replay()
        g2.replay()
    torch.cuda.synchronize()
    want, want_p = step(), project()
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(out_p, want_p)


def test_stream_argument():
    """Calls given a stream while the current one is busy: what they allocate and
    zero belongs to that stream."""
    x, r = normal((300, 2048), torch.bfloat16, 1), normal((300, 2048), torch.bfloat16, 2)
    wc, wsc = csa.fp8_quantize(normal((1024, 2048), torch.float32, 3, 2048 ** -0.5), 128)
    p = proj_inputs(300, 8, 256, 2, 512, 768, 4)
    want = csa.rmsnorm_fp8(x, r)
    want_y, want_p = csa.fp8_matmul(want[0], want[1], wc, wsc), csa.grouped_output_projection_fp8(*p)
    big = torch.randn(8192, 8192, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        (big @ big).mul_(0)                      # the current stream is busy
        got = csa.rmsnorm_fp8(x, r, stream=side)
        c, s = csa.fp8_quantize(x, stream=side)
        y = csa.fp8_matmul(got[0], got[1], wc, wsc, stream=side)
        o = csa.grouped_output_projection_fp8(*p, stream=side)
        side.synchronize()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))
        assert torch.equal(y, want_y) and torch.equal(o, want_p)
        assert torch.equal(bits(c), bits(csa.fp8_quantize(x)[0]))
    torch.cuda.synchronize()


def test_two_streams_at_once():
    cases = [operands(60, 700, 2048, 30), operands(900, 600, 1024, 31)]
    want = [csa.fp8_matmul(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = []
        for c, st in zip(cases, streams):
            with torch.cuda.stream(st):
                got.append(csa.fp8_matmul(*c))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- the layer with 8-bit projections ---------------------------------------------------

def test_layer_with_8_bit_projections():
    """One CSA layer as it is used: residual norm -> projections in FP8 (query,
    both KV groups, their logits, the indexer's operands) -> compression,
    indexer, attention -> grouped projection in FP8 -> the next norm.  Each
    8-bit stage is checked against the oracle on the GPU's own inputs to it; the
    bf16 stages in between have their own tests."""
    T, dm, H, c, m, k, n_win, g, dg = 256, 512, 64, 512, 4, 32, 128, 8, 128
    x, r = normal((T, dm), torch.bfloat16, 1), normal((T, dm), torch.bfloat16, 2)
    gain = 1 + 0.1 * normal((dm,), torch.float32, 3)
    codes, scales, h = csa.rmsnorm_fp8(x, r, gain)
    check_norm(x, r, gain, 1e-6, codes, scales)

    def project(n, seed, out=torch.bfloat16):
        w = csa.fp8_quantize(normal((n, dm), torch.float32, seed, dm ** -0.5), 128)
        y = csa.fp8_matmul(codes, scales, *w, out_dtype=out)
        check_matmul(y, codes, scales, *w)
        return y.view(1, T, n)

    q = project(H * c, 10).view(1, T, H, c)
    kv_a, kv_b, z_a, z_b = (project(c, 11 + i) for i in range(4))
    q_I = project(64 * 128, 20).view(1, T, 64, 128)
    k_I = project(128, 21)[:, :T // m].contiguous()
    w_I = project(64, 22, torch.float32)
    fmt = csa.Fmt(c=c, rope_dims=64)
    ent, win = csa.csa_compress(kv_a, kv_b, z_a, z_b, m, fmt, want_win=True)
    idx = csa.indexer_scores_topk(q_I, w_I, k_I, m, k)
    o = csa.sparse_mqa_attn(q, ent, idx, win, fmt, n_win)
    p = proj_inputs(T, H, c, g, dg, dm, 30)
    y = csa.grouped_output_projection_fp8(o[0], *p[1:])
    check_proj(y, o[0], *p[1:])
    codes2, scales2, h2 = csa.rmsnorm_fp8(y, h, gain, sum_out=h.clone())
    check_norm(y, h, gain, 1e-6, codes2, scales2)
    assert torch.equal(h2, (y.float() + h.float()).bfloat16())
