"""Host-side checks of the 8-bit projection calls that need no GPU: refusals
of the C entry points before any CUDA call, of the binding before any launch,
empty problems, and the workspace sizes."""
import ctypes

import pytest
import torch

ARG, UNSUPPORTED, WORKSPACE = 1, 2, 5
F32, BF16 = 0, 1
PTR = ctypes.c_void_p(4096)    # never dereferenced: validation fails first
MIS = ctypes.c_void_p(4104)    # not 16-byte aligned
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    from long_context_attention_csa_b200 import build, lib

    build.build()
    return lib()


def norm(L, dtype=BF16, T=4, d=256, x=PTR, x_ld=256, res=PTR, res_ld=256, gain=PTR, eps=1e-6,
         out=PTR, out_ld=256, codes=PTR, scales=PTR):
    return L.rmsnorm_fp8(dtype, T, d, x, x_ld, res, res_ld, gain, eps, out, out_ld, codes, scales,
                         None)


@pytest.mark.parametrize("change,want", [
    (dict(dtype=3), ARG), (dict(T=-1), ARG), (dict(d=0), ARG), (dict(eps=-1.0), ARG),
    (dict(eps=NAN), ARG), (dict(x=None), ARG), (dict(codes=None), ARG), (dict(scales=None), ARG),
    (dict(x=MIS), ARG), (dict(res=MIS), ARG), (dict(gain=MIS), ARG), (dict(out=MIS), ARG),
    (dict(codes=MIS), ARG), (dict(x_ld=255), ARG), (dict(x_ld=260), ARG), (dict(res_ld=248), ARG),
    (dict(out_ld=257), ARG), (dict(dtype=F32, x_ld=258), ARG), (dict(res=None), ARG),
    (dict(d=248), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
    (dict(d=32784, x_ld=32784, res_ld=32784, out_ld=32784), UNSUPPORTED),
    (dict(T=0), 0), (dict(T=0, x=None, codes=None), 0),
])
def test_rmsnorm_refusals(L, change, want):
    assert norm(L, **change) == want


def quant(L, dtype=BF16, rows=4, d=256, x=PTR, ld=256, br=1, codes=PTR, scales=PTR):
    return L.fp8_quantize(dtype, rows, d, x, ld, br, codes, scales, None)


@pytest.mark.parametrize("change,want", [
    (dict(dtype=2), ARG), (dict(rows=-1), ARG), (dict(d=0), ARG), (dict(br=0), ARG),
    (dict(br=64), ARG), (dict(x=None), ARG), (dict(x=MIS), ARG), (dict(codes=MIS), ARG),
    (dict(scales=None), ARG), (dict(ld=240), ARG), (dict(ld=257), ARG), (dict(d=250), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(d=(1 << 30) + 16, ld=(1 << 30) + 16), UNSUPPORTED),
    (dict(rows=0), 0),
])
def test_quantize_refusals(L, change, want):
    assert quant(L, **change) == want


def matmul(L, out=BF16, M=4, N=8, K=256, x=PTR, xs=PTR, w=PTR, ws_=PTR, y=PTR, ld=8, ws=PTR,
           ws_bytes=256):
    return L.fp8_matmul(out, M, N, K, x, xs, w, ws_, y, ld, ws, ws_bytes, None)


@pytest.mark.parametrize("change,want", [
    (dict(out=5), ARG), (dict(M=-1), ARG), (dict(N=-1), ARG), (dict(K=0), ARG), (dict(ld=7), ARG),
    (dict(x=None), ARG), (dict(xs=None), ARG), (dict(w=None), ARG), (dict(ws_=None), ARG),
    (dict(y=None), ARG), (dict(x=MIS), ARG), (dict(w=MIS), ARG), (dict(y=ctypes.c_void_p(4097)), ARG),
    (dict(out=F32, y=ctypes.c_void_p(4098)), ARG), (dict(K=250), UNSUPPORTED),
    (dict(M=1 << 31), UNSUPPORTED), (dict(N=1 << 31, ld=1 << 31), UNSUPPORTED),
    (dict(K=(1 << 26) + 16), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=255), WORKSPACE),
    (dict(ws=MIS), WORKSPACE), (dict(M=0), 0), (dict(N=0, ld=0), 0),
])
def test_matmul_refusals(L, change, want):
    assert matmul(L, **change) == want


def proj(L, dtype=BF16, T=4, H=8, c=64, g=2, dg=128, d=96, o=PTR, wg=PTR, wgs=PTR, wo=PTR, wos=PTR,
         y=PTR, ws=PTR, ws_bytes=1 << 40):
    return L.grouped_output_projection_fp8(dtype, T, H, c, g, dg, d, o, wg, wgs, wo, wos, y, ws,
                                           ws_bytes, None)


@pytest.mark.parametrize("change,want", [
    (dict(dtype=9), ARG), (dict(T=-1), ARG), (dict(H=0), ARG), (dict(g=0), ARG), (dict(d=0), ARG),
    (dict(o=None), ARG), (dict(wgs=None), ARG), (dict(wos=None), ARG), (dict(y=MIS), ARG),
    (dict(wg=MIS), ARG), (dict(g=3), UNSUPPORTED), (dict(g=8), UNSUPPORTED),
    (dict(dg=96), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws_bytes=3000), WORKSPACE),
    (dict(ws=MIS), WORKSPACE), (dict(T=0), 0),
])
def test_projection_refusals(L, change, want):
    assert proj(L, **change) == want


def test_workspace_sizes(L):
    from long_context_attention_csa_b200 import CSA_OP_FP8_MATMUL, CSA_OP_OUT_PROJ_FP8

    assert L.csa_workspace_bytes(CSA_OP_FP8_MATMUL, BF16, 1, 4, 0, 0, 0, 0, 0) == 256
    n = L.csa_workspace_bytes(CSA_OP_OUT_PROJ_FP8, BF16, 1, 8192, 64, 512, 8192, 0, 0)
    codes = 8192 * 32768 + 8192 * 8192          # o's and v's codes
    assert n >= 256 + codes + codes // 128      # and their scales
    assert L.csa_workspace_bytes(CSA_OP_OUT_PROJ_FP8, BF16, 1, 0, 64, 512, 8192, 0, 0) >= 256


def test_binding_refuses_cpu_tensors():
    import long_context_attention_csa_b200 as csa

    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    for call in (lambda: csa.rmsnorm_fp8(x), lambda: csa.fp8_quantize(x),
                 lambda: csa.fp8_matmul(q, s, q, s),
                 lambda: csa.grouped_output_projection_fp8(x.view(4, 4, 64), q, s, q, s)):
        with pytest.raises(csa.CSAError) as e:
            call()
        assert e.value.status == csa.CSA_E_ARG
