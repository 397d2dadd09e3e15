"""Norm with rotation where its numbers get large or small, on side streams and in graphs, and at
sizes where a warp takes several tokens."""
import pytest
import torch

from window_ref import close, norm_rope, norm_rope_backward
from trainable_block_sparse_compress_b200 import build, ops

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def cuda_library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    assert ops.device_error(clear=True) == 0
    yield
    assert ops.device_error(clear=True) == 0


def randn(g, *shape, mul=1.0):
    return (mul * torch.randn(*shape, generator=g, device="cuda")).to(BF)


def inv_freq(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


# zero rows, and rows whose norm's third power leaves fp32's range at either end
@pytest.mark.parametrize("mul,eps", [(0.0, 1e-30), (0.0, 1e-38), (1e-14, 1e-30), (1e13, 1e-6), (1e15, 1e-6)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_backward_of_tiny_and_huge_rows(mul, eps, interleaved):
    L, Hq, Hkv = 21, 4, 2
    p = ops.Params(1, Hq, Hkv)
    g = torch.Generator(device="cuda").manual_seed(7)
    x = randn(g, 1, L, Hq + 2 * Hkv, 128)
    x[:, ::2] = (x[:, ::2].float() * mul).to(BF)
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    table = ops.rope_table(p, inv_freq(64), L)
    qw, kw = (1 + 0.2 * torch.randn(128, generator=g, device="cuda") for _ in range(2))
    kwargs = dict(q_weight=qw, k_weight=kw, eps=eps, interleaved=interleaved)
    qo, ko, _ = ops.qk_norm_rope(p, q, k, v, table, **kwargs)
    dq, dk = randn(g, 1, L, Hq, 128), randn(g, 1, Hkv, L, 128)
    r = ops.qk_norm_rope_backward(p, q, k, dq, dk, dk, table, **kwargs)
    for i, (xi, w, y, d) in enumerate(((q[0], qw, qo[0], dq[0]), (k[0], kw, ko[0].transpose(0, 1), dk[0].transpose(0, 1)))):
        want, tol = norm_rope(xi, w, eps, table, interleaved)
        close(y, want, tol, "y")
        dx, tol, dw, tw = norm_rope_backward(xi, w, eps, table, interleaved, d)
        close(r[i][0], dx, tol, "dx")
        close(r[3 + i], dw, tw, "dw")
