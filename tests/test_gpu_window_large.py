"""Window attention at the sizes where its kernels take their other forms: two query tiles a CTA
with every group size and ragged lengths, split and joined keys on several streams and in graphs,
scales other than the default, and gradients against differences with a sharp bound."""
import pytest
import torch

from test_gpu_window import check_rows, inputs, randn
from window_ref import attend, attend_backward, close
from trainable_block_sparse_compress_b200 import build, ops

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def cuda_library():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    assert ops.device_error(clear=True) == 0
    yield
    assert ops.device_error(clear=True) == 0, "a kernel hit its wait time limit"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def two_tiles(B, L, Hq, Hkv):
    """256-row tiles fill the GPU: a CTA takes two query tiles."""
    rows = 256 // (Hq // Hkv)
    return (L + rows - 1) // rows * B * Hkv >= torch.cuda.get_device_properties(0).multi_processor_count


FRESH = [
    # B, L, Hq, Hkv, window, n_sink
    (1, 5000, 8, 8, 1, 0),       # the second tile starts at a later key tile than the first
    (1, 5000, 8, 8, 100, 0),
    (1, 5000, 8, 8, 300, 0),
    (1, 4999, 8, 8, 130, 5),
    (2, 3000, 8, 4, 700, 0),
    (2, 2900, 8, 4, 64, 200),
    (1, 4000, 16, 4, 5000, 0),   # plain causal
    (1, 2500, 16, 2, 257, 33),
    (1, 2400, 16, 1, 64, 0),
]


@pytest.mark.parametrize("B,L,Hq,Hkv,window,n_sink", FRESH)
def test_two_query_tiles_fresh(B, L, Hq, Hkv, window, n_sink):
    assert two_tiles(B, L, Hq, Hkv)
    q, k, v = inputs(B, L, L, Hq, Hkv, seed=L + window)
    o, lse = ops.window_attn_prefill(ops.Params(B, Hq, Hkv), q, k, v, window, n_sink)
    check_rows(o, lse, q, k, v, [L] * B, [L] * B, window, n_sink, "prefill")


RAGGED = [
    # Lq, Lmax, Hq, Hkv, window, n_sink, q_lens, kv_lens; sequences end in the first and in the second
    # tile of a CTA, at its border, or hold nothing; caches end inside a 64-key segment
    (3000, 3400, 8, 8, 100, 0, [3000, 2049, 2700, 0], [3333, 2049, 3011, 5]),
    (3000, 3400, 8, 8, 500, 70, [2688, 1, 2816], [3400, 3399, 2817]),
    (3000, 3400, 16, 4, 130, 0, [3000, 2049, 1985, 2048], [3011, 2049, 3400, 3201]),
    (3000, 3000, 16, 4, 4000, 0, [3000, 2017, 1], [3000, 2017, 1]),
    # a padded training batch: fresh sequences
    (2000, 2000, 8, 8, 300, 4, [2000, 1025, 1, 1900], [2000, 1025, 1, 1900]),
    (2000, 2000, 8, 4, 128, 0, [1999, 1985, 1, 0], [1999, 1985, 1, 0]),
    (2000, 2000, 16, 1, 200, 64, [2000, 1013, 1001], [2000, 1013, 1001]),
    (2000, 2000, 32, 4, 333, 0, [1601, 2000], [1601, 2000]),
]


@pytest.mark.parametrize("Lq,Lmax,Hq,Hkv,window,n_sink,ql,kl", RAGGED)
def test_two_query_tiles_ragged(Lq, Lmax, Hq, Hkv, window, n_sink, ql, kl):
    B = len(ql)
    assert two_tiles(B, Lq, Hq, Hkv)
    q, k, v = inputs(B, Lq, Lmax, Hq, Hkv, seed=Lmax + window)
    for b in range(B):
        q[b, ql[b]:] = NAN
        for x in (k, v):
            x[b, :, kl[b]:] = NAN
            lo = kl[b] - ql[b] - window + 1
            if lo > n_sink:
                x[b, :, n_sink:lo] = NAN
                x[b, :, (n_sink + lo) // 2] = float("inf")
    o, lse = torch.full_like(q, 7.0), torch.full((B, Hq, Lq), 7.0, device="cuda")
    ops.window_attn_chunk(ops.Params(B, Hq, Hkv), q, k, v, window, n_sink, q_lens=i32(ql), kv_lens=i32(kl), out=o, lse=lse)
    check_rows(o, lse, q, k, v, ql, kl, window, n_sink, "ragged")
    for b in range(B):
        assert (o[b, ql[b]:] == 7.0).all() and (lse[b, :, ql[b]:] == 7.0).all()


@pytest.mark.parametrize("scale", [0.02, 0.2])
def test_scales_other_than_the_default(scale):
    B, L, Hq, Hkv, W, ns = 2, 700, 8, 2, 200, 9
    p = ops.Params(B, Hq, Hkv, softmax_scale=scale)
    q, k, v = inputs(B, L, L, Hq, Hkv, seed=11)
    do = randn(torch.Generator(device="cuda").manual_seed(12), B, L, Hq, 128)
    o, lse = ops.window_attn_prefill(p, q, k, v, W, ns)
    grads = ops.window_attn_backward(p, q, k, v, o, lse, do, W, ns)
    lens = [700, 333]
    od, lsed = ops.window_attn_decode(p, q[:, 5].contiguous(), k, v, i32(lens), W, ns)
    for b in range(B):
        w, z, tw, tz = attend(q[b], k[b], v[b], 0, W, ns, scale=scale)
        close(o[b], w, tw, "o")
        close(lse[b], z, tz, "lse")
        ref, tol = attend_backward(q[b], k[b], v[b], o[b], lse[b], do[b], W, ns, scale=scale)
        for got, r, t, name in zip(grads, ref, tol, ("dq", "dk", "dv")):
            close(got[b], r, t, name)
        n = lens[b]
        w, z, tw, tz = attend(q[b, 5:6], k[b, :, :n], v[b, :, :n], n - 1, W, ns, scale=scale)
        close(od[b:b + 1], w, tw, "decode o")
        close(lsed[b][:, None], z, tz, "decode lse")


@pytest.mark.parametrize("scale", [None, 0.2])
@pytest.mark.parametrize("B,L,Hq,Hkv,W,ns", [(1, 200, 4, 2, 60, 3), (1, 300, 8, 1, 130, 0)])
def test_backward_against_differences_along_the_gradient(B, L, Hq, Hkv, W, ns, scale):
    """The kernels' gradient g against central differences of the fp64 forward, along the direction
    u = reference gradient / its norm, where the difference is the norm itself.  |u| = 1, so errors
    e of the elements move <g, u> by at most |e|: e is the elementwise bound of one rounding of P
    and dS (window_ref), plus the effect of the rounded O on D, formed here from the O at hand."""
    s = scale or 128 ** -0.5
    q, k, v = inputs(B, L, L, Hq, Hkv, seed=177)
    do = randn(torch.Generator(device="cuda").manual_seed(178), B, L, Hq, 128)
    p = ops.Params(B, Hq, Hkv, softmax_scale=scale or 0.0)
    o, lse = ops.window_attn_prefill(p, q, k, v, W, ns)
    grads = ops.window_attn_backward(p, q, k, v, o, lse, do, W, ns)
    x = [t[0].double() for t in (q, k, v)]
    d = do[0].double()
    exact_o = attend(*x, 0, W, ns, scale=scale)[0]
    ref, tol = attend_backward(q[0], k[0], v[0], exact_o, lse[0], do[0], W, ns, scale=scale)
    i = torch.arange(L, device="cuda")
    ok = (i[None] <= i[:, None]) & ((i[None] > i[:, None] - W) | (i[None] < ns))
    eff = [torch.zeros_like(t) for t in x]  # of D formed from the rounded O: dS moves by -P (D' - D)
    for h in range(Hq):
        j = h // (Hq // Hkv)
        pr = torch.exp(x[0][:, h] @ x[1][j].T * s - lse[0, h].double()[:, None]).masked_fill(~ok, 0)
        ds = pr * (d[:, h] * (o[0, :, h].double() - exact_o[:, h])).sum(-1, keepdim=True)
        eff[0][:, h] = s * ds @ x[1][j]
        eff[1][j] += s * ds.T @ x[0][:, h]

    def loss(a, b, c):
        return float((attend(a, b, c, 0, W, ns, scale=scale)[0] * d).sum())
    for n, name in enumerate(("dq", "dk", "dv")):
        norm = float(ref[n].norm())
        u = ref[n] / norm
        h = 1e-5
        lo, hi = ([t + f * u if m == n else t for m, t in enumerate(x)] for f in (-h, h))
        want = (loss(*hi) - loss(*lo)) / (2 * h)
        assert abs(want - norm) <= 1e-5 * norm, f"{name}: the reference itself"  # third derivatives x h^2
        bound = float(tol[n].norm() + eff[n].norm()) + 1e-4 * abs(want)
        assert bound < 0.1 * abs(want), f"{name}: the bound is not sharp"
        got = float((grads[n][0].double() * u).sum())
        assert abs(got - want) <= bound, f"{name}: {got} against {want}"


def split_calls(seed):
    """Calls whose keys are split and joined: chunk (workspace), decode (cluster; workspace), backward
    (cut key tiles).  Returns their inputs and the calls."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    pc, pd, pw, pb = ops.Params(1, 16, 1), ops.Params(2, 8, 2), ops.Params(1, 8, 1), ops.Params(1, 8, 1)
    t = dict(qc=randn(g, 1, 7, 16, 128), kc=randn(g, 1, 1, 20000, 128), vc=randn(g, 1, 1, 20000, 128),
             qd=randn(g, 2, 8, 128), kd=randn(g, 2, 2, 3000, 128), vd=randn(g, 2, 2, 3000, 128),
             qw=randn(g, 1, 8, 128), kw=randn(g, 1, 1, 70000, 128), vw=randn(g, 1, 1, 70000, 128),
             qb=randn(g, 1, 2000, 8, 128), kb=randn(g, 1, 1, 2000, 128), vb=randn(g, 1, 1, 2000, 128),
             do=randn(g, 1, 2000, 8, 128), ld=i32([3000, 1777]), lw=i32([70000 - seed]))

    def run():
        oc = ops.window_attn_chunk(pc, t["qc"], t["kc"], t["vc"], 100000)
        od = ops.window_attn_decode(pd, t["qd"], t["kd"], t["vd"], t["ld"], 3000)
        ow = ops.window_attn_decode(pw, t["qw"], t["kw"], t["vw"], t["lw"], 70000)
        ob = ops.window_attn_prefill(pb, t["qb"], t["kb"], t["vb"], 2000, 3)
        gb = ops.window_attn_backward(pb, t["qb"], t["kb"], t["vb"], *ob, t["do"], 2000, 3)
        return (*oc, *od, *ow, *ob, *gb)
    return t, run


def test_split_calls_on_streams_at_once():
    (_, run1), (_, run2) = split_calls(1), split_calls(2)
    want1, want2 = run1(), run2()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        for s, run, want in ((s1, run1, want1), (s2, run2, want2)):
            with torch.cuda.stream(s):
                got.append((run(), want))
    torch.cuda.synchronize()
    for res, want in got:
        assert all(torch.equal(a, b) for a, b in zip(res, want))


def test_split_calls_in_a_graph():
    t, run = split_calls(3)
    t2, run2 = split_calls(4)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    want2 = run2()
    for name in t:
        t[name].copy_(t2[name])
    for _ in range(3):
        for x in out:
            x.fill_(NAN)
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want2))


def test_a_workspace_with_gaps_is_refused():
    q, k, v = inputs(1, 7, 20000, 16, 1, seed=1)
    p = ops.Params(1, 16, 1)
    for ws in (torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 26),
               torch.empty(1 << 27, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="ws must be contiguous"):
            ops.window_attn_chunk(p, q, k, v, 100000, ws=ws)
    want = ops.window_attn_chunk(p, q, k, v, 100000)
    for n in (1, 1 << 26):  # one too small is replaced
        got = ops.window_attn_chunk(p, q, k, v, 100000, ws=torch.empty(n, dtype=torch.uint8, device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_longest_sequence_forward_and_backward():
    """The last tokens of 262144: they see the last keys only, so a slice of them is the whole reference."""
    L, Hq, Hkv, W, n = 262144, 4, 2, 300, 500
    q, k, v = inputs(1, L, L, Hq, Hkv, seed=9)
    do = randn(torch.Generator(device="cuda").manual_seed(10), 1, L, Hq, 128)
    p = ops.Params(1, Hq, Hkv)
    o, lse = ops.window_attn_prefill(p, q, k, v, W)
    dq, dk, dv = ops.window_attn_backward(p, q, k, v, o, lse, do, W)
    m = n + W  # tokens of the slice; its last n have all of their keys and queries in it
    qs, os_, ds = (x[0, -m:] for x in (q, o, do))
    ks, vs, ls = k[0, :, -m:], v[0, :, -m:], lse[0, :, -m:]
    w, z, tw, tz = attend(qs, ks, vs, 0, W, 0)
    close(o[0, -n:], w[-n:], tw[-n:], "o")
    close(lse[0, :, -n:], z[:, -n:], tz[:, -n:], "lse")
    ref, tol = attend_backward(qs, ks, vs, os_, ls, ds, W, 0)
    close(dq[0, -n:], ref[0][-n:], tol[0][-n:], "dq")
    for got, r, t, name in ((dk, ref[1], tol[1], "dk"), (dv, ref[2], tol[2], "dv")):
        close(got[0, :, -n:], r[:, -n:], t[:, -n:], name)
