"""A launch that the runtime refuses is reported by its own call and by no later one."""
import contextlib
import ctypes

import pytest
import torch

from trainable_block_sparse_compress_b200 import _lib, build, ops

pytestmark = pytest.mark.gpu


@contextlib.contextmanager
def refusing_stream():
    """A stream whose capture has been invalidated: every launch on it is refused on the host."""
    rt = ctypes.CDLL("libcudart.so.12")  # the one torch has loaded
    s, graph = ctypes.c_void_p(), ctypes.c_void_p()
    assert rt.cudaStreamCreateWithFlags(ctypes.byref(s), 1) == 0
    assert rt.cudaStreamBeginCapture(s, 2) == 0
    assert rt.cudaStreamSynchronize(s) != 0  # not allowed in a capture
    rt.cudaGetLastError()
    try:
        yield s.value
    finally:
        assert rt.cudaStreamEndCapture(s, ctypes.byref(graph)) != 0 and not graph.value
        rt.cudaGetLastError()
        assert rt.cudaStreamDestroy(s) == 0


def test_a_refused_cluster_launch_is_not_reported_by_the_next_call():
    build.build()
    B, Hq, Hkv, Lmax = 2, 8, 2, 3000
    p = ops.Params(B, Hq, Hkv, topk=8)
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(B, Hq, 128, generator=g, device="cuda").bfloat16()
    k, v = (torch.randn(B, Hkv, Lmax, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    lens = torch.tensor([Lmax, 1234], dtype=torch.int32, device="cuda")
    kc = ops.compress_keys(p, k)
    want = ops.window_attn_decode(p, q, k, v, lens, Lmax)  # chunks joined in a cluster
    want_step = ops.decode_step(p, q, k, v, kc, lens)
    out, lse = torch.zeros_like(q), torch.zeros(B, Hq, device="cuda")
    idx = torch.zeros(B, Hkv, 1, 8, dtype=torch.int32, device="cuda")
    ws = torch.empty(ops.workspace_size(p, _lib.OP_WINDOW_DECODE, Lmax), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()

    def refused_window(stream):
        return _lib.load().infllmv2_window_attn_decode(
            ctypes.byref(p.c()), q.data_ptr(), k.data_ptr(), v.data_ptr(), lens.data_ptr(), Lmax, Lmax, 0,
            out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), stream)

    def refused_step(stream):
        return _lib.load().infllmv2_decode_step(
            ctypes.byref(p.c()), q.data_ptr(), None, None, k.data_ptr(), v.data_ptr(), kc.data_ptr(), lens.data_ptr(),
            None, Lmax, idx.data_ptr(), out.data_ptr(), lse.data_ptr(), stream)
    with refusing_stream() as stream:
        for refused in (refused_window, refused_step):
            assert refused(stream) == _lib.ERR_CUDA
            assert all(torch.equal(a, b) for a, b in zip(ops.window_attn_decode(p, q, k, v, lens, Lmax), want))
            assert refused(stream) == _lib.ERR_CUDA
            assert all(torch.equal(a, b) for a, b in zip(ops.decode_step(p, q, k, v, kc, lens), want_step))
            assert refused(stream) == _lib.ERR_CUDA
            assert torch.equal(ops.compress_keys(p, k), kc)
    torch.cuda.synchronize()
    assert (out == 0).all() and (lse == 0).all() and ops.device_error(clear=True) == 0
