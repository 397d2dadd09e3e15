"""Host-side refusals of the norm-and-rotation and window-attention calls: nothing is launched."""
import ctypes
import math

import pytest

from trainable_block_sparse_compress_b200 import _lib, build
from trainable_block_sparse_compress_b200.ops import Params

GOOD, OTHER = 4096, 8192  # fake 16-byte aligned "device addresses": never dereferenced
INV, UNS, WS = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED, _lib.ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def cp(**kw):
    return ctypes.byref(Params(**{**dict(batch=2, num_q_heads=8, num_kv_heads=2, topk=16), **kw}).c())


def variants(base, changes):
    for i, val in changes:
        args = list(base)
        args[i] = val
        yield i, val, args


def test_window_attn_refusals(lib):
    f = lib.infllmv2_window_attn
    # q, Lq, k, v, q_lens, kv_lens, Lmax, window, n_sink, o, lse, ws, ws_bytes, stream
    base = [GOOD, 8, GOOD, GOOD, None, None, 128, 16, 4, GOOD, None, GOOD, 1 << 40, None]
    changes = [(i, None) for i in (0, 2, 3, 9)] + [(i, GOOD + 8) for i in (0, 2, 3, 9)] + [
        (1, 0), (1, 129), (6, 0), (6, _lib.MAX_SEQ_LEN + 1), (4, GOOD + 2), (5, GOOD + 1), (7, 0), (7, -4), (8, -1),
        (10, GOOD + 2)]
    for i, val, args in variants(base, changes):
        assert f(cp(), *args) == INV, (i, val)
    assert f(None, *base) == INV
    assert f(cp(head_dim=64), *base) == UNS
    assert f(cp(num_q_heads=6), *base) == UNS  # a group of 3
    need = lib.infllmv2_workspace_size(cp(), _lib.OP_WINDOW_ATTN, 8)
    assert need != ctypes.c_size_t(-1).value
    if need:
        for ws, n in ((None, 0), (GOOD, need - 1), (GOOD + 8, need)):
            assert f(cp(), *base[:11], ws, n, None) == WS
    big = Params(batch=1 << 15, num_q_heads=8, num_kv_heads=2, topk=16)  # 2^15 x 262144 rows
    assert f(ctypes.byref(big.c()), *base[:6], _lib.MAX_SEQ_LEN, *base[7:]) == UNS


def test_window_decode_refusals(lib):
    f = lib.infllmv2_window_attn_decode
    # q, k, v, lens, Lmax, window, n_sink, o, lse, ws, ws_bytes, stream
    base = [GOOD, GOOD, GOOD, GOOD, 128, 16, 4, GOOD, None, GOOD, 1 << 40, None]
    changes = [(i, None) for i in (0, 1, 2, 3, 7)] + [(i, GOOD + 8) for i in (0, 1, 2, 7)] + [
        (3, GOOD + 2), (4, 0), (4, _lib.MAX_SEQ_LEN + 1), (5, 0), (6, -1), (8, GOOD + 1)]
    for i, val, args in variants(base, changes):
        assert f(cp(), *args) == INV, (i, val)
    assert f(cp(block_size=32), *base) == UNS
    need = lib.infllmv2_workspace_size(cp(), _lib.OP_WINDOW_DECODE, 128)
    assert need != ctypes.c_size_t(-1).value
    if need:
        for ws, n in ((None, 0), (GOOD, need - 1), (GOOD + 8, need)):
            assert f(cp(), *base[:9], ws, n, None) == WS


def test_window_backward_refusals(lib):
    f = lib.infllmv2_window_attn_backward
    # q, k, v, o, lse, d_o, lens, L, window, n_sink, dq, dk, dv, ws, ws_bytes, stream
    base = [GOOD] * 6 + [None, 128, 16, 4, GOOD, GOOD, GOOD, GOOD, 1 << 40, None]
    ptrs = (0, 1, 2, 3, 4, 5, 10, 11, 12)
    changes = [(i, None) for i in ptrs] + [(i, GOOD + 8) for i in ptrs if i != 4] + [
        (4, GOOD + 2), (6, GOOD + 2), (7, 0), (7, _lib.MAX_SEQ_LEN + 1), (8, 0), (9, -1)]
    for i, val, args in variants(base, changes):
        assert f(cp(), *args) == INV, (i, val)
    assert f(cp(kernel_size=16), *base) == UNS
    need = lib.infllmv2_workspace_size(cp(), _lib.OP_WINDOW_BACKWARD, 128)
    assert need != ctypes.c_size_t(-1).value
    if need:
        for ws, n in ((None, 0), (GOOD, need - 1), (GOOD + 8, need)):
            assert f(cp(), *base[:13], ws, n, None) == WS


def test_qk_norm_rope_refusals(lib):
    f = lib.infllmv2_qk_norm_rope
    # q, qs, k, ks, v, vs, Lq, qw, kw, fp32, eps, table, rows, rot, interleaved, starts, q_lens, q_out, k_out, v_out,
    # Lout, at_position, lens_out, stream
    base = [GOOD, 1024, GOOD, 256, GOOD, 256, 4, GOOD, GOOD, 0, 1e-6, GOOD, 64, 128, 0, GOOD, GOOD, GOOD, GOOD, GOOD,
            64, 1, OTHER, None]
    ptrs = (0, 2, 4, 11, 17, 18, 19)
    changes = [(i, None) for i in ptrs] + [(i, GOOD + 8) for i in ptrs + (7, 8)] + [
        (1, 1016), (1, 1028), (3, 0), (3, 252), (5, 128), (5, 260), (6, 0), (9, 2), (10, 0.0), (10, -1.0),
        (10, math.inf), (10, math.nan), (12, 0), (12, _lib.MAX_SEQ_LEN + 1), (13, 0), (13, 8), (13, 120), (13, 144),
        (14, 2), (15, GOOD + 2), (16, GOOD + 2), (20, 0), (21, 2), (22, GOOD + 1), (22, GOOD)]
    for i, val, args in variants(base, changes):
        assert f(cp(), *args) == INV, (i, val)
    fresh = list(base)
    fresh[20], fresh[21] = 3, 0  # fewer output rows than tokens
    assert f(cp(), *fresh) == INV
    assert f(cp(head_dim=64), *base) == UNS


def test_qk_norm_rope_backward_refusals(lib):
    f = lib.infllmv2_qk_norm_rope_backward
    # q, qs, k, ks, d_q, d_k, d_v, Lq, qw, kw, fp32, eps, table, rows, rot, interleaved, starts, q_lens, dq, dqs, dk,
    # dks, dv, dvs, d_qw, d_kw, ws, ws_bytes, stream
    need = lib.infllmv2_workspace_size(cp(), _lib.OP_QK_NORM_ROPE_BACKWARD, 4)
    assert 0 < need != ctypes.c_size_t(-1).value
    base = [GOOD, 1024, GOOD, 256, GOOD, GOOD, GOOD, 4, GOOD, GOOD, 1, 1e-6, GOOD, 64, 64, 1, None, None, GOOD, 1536,
            GOOD, 1536, GOOD, 1536, GOOD, GOOD, GOOD, need, None]
    ptrs = (0, 2, 4, 5, 6, 12, 18, 20, 22)
    changes = [(i, None) for i in ptrs] + [(i, GOOD + 8) for i in ptrs + (8, 9)] + [
        (19, 1016), (21, 128), (23, 260), (24, GOOD + 2), (25, GOOD + 1), (11, 0.0), (14, 24), (16, GOOD + 2)]
    for i, val, args in variants(base, changes):
        assert f(cp(), *args) == INV, (i, val)
    for i, val, args in variants(base, [(26, None), (27, need - 1), (26, GOOD + 8)]):
        assert f(cp(), *args) == WS, (i, val)


def test_rope_table_refusals(lib):
    f = lib.infllmv2_rope_table
    base = [GOOD, 128, 100, 1.0, GOOD, None]  # inv_freq, rot, n, scale, table, stream
    for i, val, args in variants(base, [(0, None), (4, None), (0, GOOD + 2), (4, GOOD + 8), (1, 0), (1, 20), (1, 256),
                                        (2, 0), (2, _lib.MAX_SEQ_LEN + 1), (3, math.nan), (3, math.inf)]):
        assert f(cp(), *args) == INV, (i, val)
