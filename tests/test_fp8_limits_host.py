"""Limits of the 8-bit products that need no GPU: columns of one sum."""
import pytest

from test_fp8_host import BF16, F32, UNSUPPORTED, WORKSPACE, L, matmul, proj  # noqa: F401

ONE_SUM = 1 << 17    # columns of one tensor-core sum, where the result is bf16 or E4M3


@pytest.mark.parametrize("out,K,want", [
    (BF16, ONE_SUM, WORKSPACE), (BF16, ONE_SUM + 16, UNSUPPORTED), (BF16, 1 << 26, UNSUPPORTED),
    (F32, ONE_SUM + 16, WORKSPACE), (F32, 1 << 26, WORKSPACE), (F32, (1 << 26) + 16, UNSUPPORTED),
])
def test_matmul_columns_of_one_sum(L, out, K, want):
    """Accepted calls go on to the workspace check, which ends them here."""
    assert matmul(L, out=out, K=K, ws=None) == want


@pytest.mark.parametrize("change,want", [
    (dict(H=4, c=1 << 16, g=2), WORKSPACE),                  # a group of 2^17 columns
    (dict(H=4, c=1 << 16, g=1), UNSUPPORTED),
    (dict(H=2, c=ONE_SUM + 128, g=2), UNSUPPORTED),
    (dict(g=8, H=8, c=128, dg=1 << 14), WORKSPACE),          # g d_g = 2^17
    (dict(g=8, H=8, c=128, dg=(1 << 14) + 128), UNSUPPORTED),
])
def test_projection_columns_of_one_sum(L, change, want):
    assert proj(L, ws=None, **change) == want


def test_a_large_workspace_of_the_calls_own_is_zeroed_at_its_status_word_only(monkeypatch):
    import torch

    import long_context_attention_csa_b200 as csa

    asked = []

    def workspace(nbytes, device=None):
        asked.append(nbytes)
        return torch.zeros(max(nbytes, 256), dtype=torch.uint8)

    monkeypatch.setattr(csa, "workspace", workspace)
    for n in (256, 4096, 16 << 20, (16 << 20) + 256, 64 << 20):
        address, size, ws = csa._ws(None, n, 0)
        assert address == ws.data_ptr() and size == ws.numel() >= n
        assert int(ws[:256].max()) == 0
    assert max(asked) <= 16 << 20
