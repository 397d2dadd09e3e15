"""Padded batches through the norm with rotation and the window attention when the calls make
their own outputs: no row of them may hold what was in memory before."""
import pytest
import torch

from trainable_block_sparse_compress_b200 import build, ops

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
B, L, HQ, HKV = 3, 700, 8, 2
LENS = [700, 1, 333]


@pytest.fixture(scope="module", autouse=True)
def cuda_library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    assert ops.device_error(clear=True) == 0
    yield
    assert ops.device_error(clear=True) == 0


def poison():
    """Leaves NaN in the allocator's free blocks of every size up to a few MB."""
    del_me = [torch.full((n,), float("nan"), dtype=BF, device="cuda") for n in
              [1 << i for i in range(6, 24)] * 4 + [B * L * h * 128 for h in (HQ, HKV, HQ + 2 * HKV)] * 8]
    torch.cuda.synchronize()
    del del_me


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(BF)


def padding(x):
    """The padded rows of [B, L, H, d]."""
    return torch.cat([x[b, LENS[b]:].flatten() for b in range(B)])


def test_gradients_of_padding_are_zero_in_tensors_made_by_the_calls():
    g = torch.Generator(device="cuda").manual_seed(1)
    p = ops.Params(B, HQ, HKV)
    q, do = randn(g, B, L, HQ, 128), randn(g, B, L, HQ, 128)
    k, v = randn(g, B, HKV, L, 128), randn(g, B, HKV, L, 128)
    lens = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    o, lse = ops.window_attn_chunk(p, q, k, v, 100, 4, q_lens=lens, kv_lens=lens, out=torch.zeros_like(q))
    poison()
    dq, dk, dv = ops.window_attn_backward(p, q, k, v, o, lse, do, 100, 4, lens=lens)
    for x in (dq, dk.transpose(1, 2), dv.transpose(1, 2)):
        assert (padding(x) == 0).all()
    table = ops.rope_table(p, 1e4 ** (-torch.arange(64, device="cuda") / 64), L)
    w = torch.ones(128, device="cuda")
    x = randn(g, B, L, HQ + 2 * HKV, 128)
    poison()
    r = ops.qk_norm_rope_backward(p, x[:, :, :HQ], x[:, :, HQ:HQ + HKV], dq, dk, dv, table, w, w, q_lens=lens)
    for y in r[:3]:
        assert (padding(y) == 0).all()
    # what a training step does next: the projection's weight gradient over all rows
    packed = torch.cat(r[:3], 2).view(B * L, -1)
    assert torch.isfinite(packed.T.float() @ torch.ones(B * L, 16, device="cuda")).all()


def test_forward_rows_of_padding_are_zero_in_tensors_made_by_the_calls():
    g = torch.Generator(device="cuda").manual_seed(2)
    p = ops.Params(B, HQ, HKV)
    lens = torch.tensor(LENS, dtype=torch.int32, device="cuda")
    table = ops.rope_table(p, 1e4 ** (-torch.arange(64, device="cuda") / 64), L)
    x = randn(g, B, L, HQ + 2 * HKV, 128)
    poison()
    q, k, v = ops.qk_norm_rope(p, x[:, :, :HQ], x[:, :, HQ:HQ + HKV], x[:, :, HQ + HKV:], table, q_lens=lens)
    for y in (q, k.transpose(1, 2), v.transpose(1, 2)):
        assert (padding(y) == 0).all()
    poison()
    o, _ = ops.window_attn_chunk(p, q, k, v, 100, 4, q_lens=lens, kv_lens=lens)
    assert (padding(o) == 0).all()
    # the same rows as in tensors of the caller, whose padding is left alone
    mine = [torch.full_like(y, 7.0) for y in (q, k, v, o)]
    ops.qk_norm_rope(p, x[:, :, :HQ], x[:, :, HQ:HQ + HKV], x[:, :, HQ + HKV:], table, q_lens=lens, q_out=mine[0],
                     k_out=mine[1], v_out=mine[2])
    ops.window_attn_chunk(p, mine[0], mine[1], mine[2], 100, 4, q_lens=lens, kv_lens=lens, out=mine[3])
    for got, m in zip((q, k.transpose(1, 2), v.transpose(1, 2), o),
                      (mine[0], mine[1].transpose(1, 2), mine[2].transpose(1, 2), mine[3])):
        assert (padding(m) == 7.0).all()
        for b in range(B):
            assert torch.equal(got[b, :LENS[b]], m[b, :LENS[b]])
