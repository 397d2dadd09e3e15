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


def projection(g, B, L, Hq, Hkv):
    x = randn(g, B, L, Hq + 2 * Hkv, 128, mul=2.0)
    return x, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]


# so many tokens that a warp of the forward takes several pairs of them
@pytest.mark.parametrize("L,Hq,Hkv,interleaved,n,t0", [
    (32001, 32, 32, False, [32001], [0]),
    (16001, 32, 32, True, [16001, 9001], [3, 0]),
    (65001, 32, 2, False, [65001], [7])])
def test_forward_with_several_tokens_a_warp(L, Hq, Hkv, interleaved, n, t0):
    B, rot = len(n), 128
    p = ops.Params(B, Hq, Hkv)
    g = torch.Generator(device="cuda").manual_seed(L)
    _, q, k, v = projection(g, B, L, Hq, Hkv)
    qw, kw = (1 + 0.2 * torch.randn(128, generator=g, device="cuda") for _ in range(2))
    Lmax = L + 16
    table = ops.rope_table(p, inv_freq(rot), Lmax)
    cache = [torch.full((B, Hkv, Lmax, 128), 7.0, dtype=BF, device="cuda") for _ in range(2)]
    qo = torch.full((B, L, Hq, 128), 7.0, dtype=BF, device="cuda")
    starts, q_lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (t0, n))
    lens = torch.empty_like(starts)
    ops.qk_norm_rope(p, q, k, v, table, qw, kw, interleaved=interleaved, starts=starts, q_lens=q_lens,
                     k_cache=cache[0], v_cache=cache[1], q_out=qo, lens_out=lens)
    assert lens.tolist() == [a + b for a, b in zip(t0, n)]
    for b in range(B):
        at = slice(t0[b], t0[b] + n[b])
        for r in range(0, n[b], 8192):
            e = min(n[b], r + 8192)
            for got, x, w, name in ((qo[b, r:e], q, qw, "q"),
                                    (cache[0][b, :, t0[b] + r:t0[b] + e].transpose(0, 1), k, kw, "k")):
                want, tol = norm_rope(x[b, r:e], w, 1e-6, table[t0[b] + r:t0[b] + e], interleaved)
                close(got, want, tol, name)
        assert torch.equal(cache[1][b, :, at].transpose(0, 1), v[b, :n[b]])
        assert (qo[b, n[b]:] == 7.0).all()
        for c in cache:
            assert (c[b, :, :t0[b]] == 7.0).all() and (c[b, :, t0[b] + n[b]:] == 7.0).all()


def test_on_two_streams_and_in_a_graph():
    B, L, Hq, Hkv, Lmax = 3, 50, 8, 2, 400
    p = ops.Params(B, Hq, Hkv)
    table = ops.rope_table(p, inv_freq(128), Lmax)
    w = torch.ones(128, device="cuda")

    def make(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        t = dict(x=projection(g, B, L, Hq, Hkv)[0], one=projection(g, B, 1, Hq, Hkv)[0],
                 starts=torch.randint(0, 300, (B,), generator=g, device="cuda", dtype=torch.int32),
                 q_lens=torch.randint(1, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32),
                 dq=randn(g, B, L, Hq, 128), dk=randn(g, B, Hkv, L, 128), dv=randn(g, B, Hkv, L, 128))

        def run():
            def views(x):
                return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
            kc, vc = torch.zeros(B, Hkv, Lmax, 128, dtype=BF, device="cuda"), \
                torch.zeros(B, Hkv, Lmax, 128, dtype=BF, device="cuda")
            lens, lens2 = torch.empty_like(t["starts"]), torch.empty_like(t["starts"])
            q1, _, _ = ops.qk_norm_rope(p, *views(t["x"]), table, w, w, starts=t["starts"], q_lens=t["q_lens"],
                                        k_cache=kc, v_cache=vc, lens_out=lens)
            # the next token, right behind the chunk: it needs the lengths that the call before wrote
            q2, _, _ = ops.qk_norm_rope(p, *views(t["one"]), table, w, w, starts=lens, k_cache=kc, v_cache=vc,
                                        lens_out=lens2)
            q, k, _ = views(t["x"])
            r = ops.qk_norm_rope_backward(p, q, k, t["dq"], t["dk"], t["dv"], table, w, w, starts=t["starts"],
                                          q_lens=t["q_lens"])
            return (q1, q2, kc, vc, lens, lens2, *r)
        return t, run
    (t1, run1), (t2, run2) = make(1), make(2)
    want1, want2 = run1(), run2()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        for s, run, want in ((s1, run1, want1), (s2, run2, want2)):
            with torch.cuda.stream(s):
                got.append((run(), want))
    torch.cuda.synchronize()
    for res, want in got:
        assert all(torch.equal(a, b) for a, b in zip(res, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run1()
    for name in t1:
        t1[name].copy_(t2[name])
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want2))
    assert want2[5].tolist() == (t2["starts"] + t2["q_lens"] + 1).tolist()
