"""Host-side checks of the binding for the norm-and-rotation and window-attention calls: they
come before any CUDA call, so they are tested with tensors of the host."""
import ctypes
import os
import re

import pytest
import torch

from trainable_block_sparse_compress_b200 import _lib, build, ops

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def library():
    build.build()


def window_calls(window, n_sink):
    p = ops.Params(1, 4, 2)
    q, k = torch.zeros(1, 8, 4, 128, dtype=BF), torch.zeros(1, 2, 8, 128, dtype=BF)
    lse, lens = torch.zeros(1, 4, 8), torch.ones(1, dtype=torch.int32)
    yield lambda: ops.window_attn_prefill(p, q, k, k, window, n_sink)
    yield lambda: ops.window_attn_chunk(p, q, k, k, window, n_sink)
    yield lambda: ops.window_attn_decode(p, q[:, 0], k, k, lens, window, n_sink)
    yield lambda: ops.window_attn_backward(p, q, k, k, q, lse, q, window, n_sink)


# each of them is a legal number once cut to 32 bits
@pytest.mark.parametrize("window,n_sink", [(2**32 + 4096, 0), (-(2**32) + 5, 0), (4, 2**32), (4, 2**40 + 1),
                                           (2**33 + 1, 2**33), (4, -(2**32))])
def test_numbers_past_32_bits_are_refused_not_cut(window, n_sink):
    for call in window_calls(window, n_sink):
        with pytest.raises(_lib.InfLLMv2Error, match="invalid argument"):
            call()


def test_largest_numbers_pass_the_check():
    for call in window_calls(2**31 - 1, 2**31 - 1):
        with pytest.raises(ValueError, match="CUDA tensor"):  # the next check
            call()


def test_sizes_past_32_bits_are_refused_not_cut():
    p = ops.Params(1, 4, 2)
    with pytest.raises(_lib.InfLLMv2Error, match="invalid argument"):
        ops.workspace_size(p, _lib.OP_WINDOW_BACKWARD, 2**32 + 100)
    for field in ("batch", "num_q_heads", "topk", "n_init", "n_local", "score_mode", "pool_mode"):
        good = dict(batch=1, num_q_heads=4, num_kv_heads=2, topk=16)
        ops.Params(**good).c()
        bad = {**good, field: 2**32 + good.get(field, 0)}
        with pytest.raises(_lib.InfLLMv2Error, match="invalid argument"):
            ops.Params(**bad).c()


@pytest.mark.parametrize("ws", [torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1, dtype=torch.uint8).expand(1 << 20)])
@pytest.mark.parametrize("op", [_lib.OP_SELECT_DECODE, _lib.OP_ATTN_DECODE, _lib.OP_ATTN_BACKWARD,
                                _lib.OP_QK_NORM_ROPE_BACKWARD, _lib.OP_WINDOW_ATTN, _lib.OP_WINDOW_DECODE,
                                _lib.OP_WINDOW_BACKWARD])
def test_a_workspace_of_the_host_is_refused(ws, op):
    # the kernels would write to its address
    with pytest.raises(ValueError, match="ws must be a CUDA tensor"):
        ops._workspace(ops.Params(1, 4, 2), op, 100, ws, torch.empty(1))


# The copying thread of each window kernel: a copy that lands after its CTA has ended writes into
# the next CTA's shared memory.  No timeout is provoked on the GPU; the sources are read instead.
COPIERS = [("window_tc.cuh", "window_tc_kernel"), ("window_bwd_tc.cuh", "window_dkdv"), ("window_bwd_tc.cuh", "window_dq"),
           ("window_decode.cuh", "window_decode_kernel")]


@pytest.mark.parametrize("file,fn", COPIERS)
def test_copying_threads_wait_for_every_copy_before_they_return(file, fn):
    src = open(os.path.join(build.CSRC, file)).read()
    body = src[re.search(rf"\n\s*(__device__ __forceinline__ void )?{fn}\(", src).start():]
    body = body[:body.index("\n}\n")]
    armed = set(re.findall(r"mbar_arrive_expect_tx\(&S\.(\w+)", body))
    for either in re.findall(r"uint64_t\* bar = any \? &S\.(.*?) : &S\.(\w+)", body):
        armed |= {re.sub(r"\[0\]$", "", either[0]), either[1]}
    assert armed, "the kernel arms no barrier"
    last = max(m.end() for m in re.finditer(r"tma_load_\dd\(", body))
    tail = body[last:]
    tail = tail[:re.search(r"\n    return;|__syncwarp\(\);\n  \}", tail).end()]
    assert "if (S.abort && lane == 0)" not in tail, "waits for its copies only when a wait has been given up already"
    waited = {re.sub(r"\[0\]$|\[x\]$", "", x) for x in re.findall(r"mbar_wait_drain\(&S\.([\w\[\]]+)", tail)}
    waited |= set(re.findall(r"drain_ring\(S\.(\w+)", tail))
    assert waited == armed


# dq, dk and dv are written while other CTAs still read the inputs: in place would be a race
@pytest.mark.parametrize("out,other", [(o, i) for o in ("dq", "dk", "dv") for i in ("q", "k", "v", "d_o")] + [
    ("dk", "dq"), ("dv", "dq"), ("dv", "dk")])
@pytest.mark.parametrize("shift", [0, -256, 256])
def test_window_backward_in_place_is_refused(out, other, shift):
    p = ops.Params(2, 8, 2)
    # addresses far apart, never read: nothing is launched
    at = {n: (i + 1) << 24 for i, n in enumerate(("q", "k", "v", "o", "lse", "d_o", "dq", "dk", "dv", "ws"))}
    at[out] = at[other] + shift
    st = _lib.load().infllmv2_window_attn_backward(
        ctypes.byref(p.c()), at["q"], at["k"], at["v"], at["o"], at["lse"], at["d_o"], None, 128, 16, 4, at["dq"],
        at["dk"], at["dv"], at["ws"], 1 << 40, None)
    assert st == _lib.ERR_INVALID_ARG


@pytest.mark.parametrize("which", ["starts", "q_lens"])
def test_norm_rope_lengths_in_place_are_refused(which):
    # other CTAs still read them when the new lengths are written
    p = ops.Params(2, 8, 2)
    at = {n: (i + 1) << 24 for i, n in enumerate(("q", "k", "v", "table", "starts", "q_lens", "qo", "ko", "vo"))}
    st = _lib.load().infllmv2_qk_norm_rope(
        ctypes.byref(p.c()), at["q"], 1024, at["k"], 256, at["v"], 256, 4, None, None, 0, 1e-6, at["table"], 64, 128, 0,
        at["starts"], at["q_lens"], at["qo"], at["ko"], at["vo"], 64, 1, at[which], None)
    assert st == _lib.ERR_INVALID_ARG
