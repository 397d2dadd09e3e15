"""Window attention (prefill, chunk, decode, backward) against the fp64 reference."""
import pytest
import torch

from window_ref import attend, attend_backward, close
from trainable_block_sparse_compress_b200 import _lib, build, ops

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


def randn(g, *shape, mul=1.0):
    return (mul * torch.randn(*shape, generator=g, device="cuda")).to(BF)


def inputs(B, Lq, Lmax, Hq, Hkv, seed, mul=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (randn(g, B, Lq, Hq, 128, mul=mul), randn(g, B, Hkv, Lmax, 128, mul=mul), randn(g, B, Hkv, Lmax, 128))


def check_rows(o, lse, q, k, v, ql, kl, window, n_sink, what):
    """o [B, Lq, Hq, d], lse [B, Hq, Lq]: rows 0..ql[b]-1 of every sequence."""
    for b in range(q.shape[0]):
        n, N = ql[b], kl[b]
        if n == 0:
            continue
        w, z, tw, tz = attend(q[b, :n], k[b, :, :N], v[b, :, :N], N - n, window, n_sink)
        close(o[b, :n], w, tw, f"{what} o[{b}]")
        if lse is not None:
            close(lse[b, :, :n], z, tz, f"{what} lse[{b}]")


PREFILL = [
    # B, L, Hq, Hkv, window, n_sink
    (1, 1, 1, 1, 1, 0),
    (1, 64, 16, 1, 16, 4),
    (2, 129, 8, 1, 64, 1),
    (1, 517, 32, 2, 128, 64),
    (1, 1000, 4, 4, 333, 0),
    (1, 1030, 2, 1, 1, 0),          # every query sees its own key only
    (1, 1030, 4, 2, 1, 3),
    (1, 700, 8, 2, 10000, 0),       # plain causal
    (1, 700, 16, 1, 2147483647, 2147483647),
    (1, 300, 16, 1, 20, 500),       # sinks past the end: plain causal
    (2, 2051, 4, 2, 256, 100),
    (3, 385, 2, 2, 64, 65),
    (1, 5000, 32, 2, 1000, 70),
]


@pytest.mark.parametrize("B,L,Hq,Hkv,window,n_sink", PREFILL)
def test_prefill_matches_reference(B, L, Hq, Hkv, window, n_sink):
    q, k, v = inputs(B, L, L, Hq, Hkv, seed=L + window % 1000)
    p = ops.Params(B, Hq, Hkv)
    o, lse = ops.window_attn_prefill(p, q, k, v, window, n_sink)
    check_rows(o, lse, q, k, v, [L] * B, [L] * B, window, n_sink, "prefill")
    o2, none = ops.window_attn_prefill(p, q, k, v, window, n_sink, want_lse=False)
    assert none is None and torch.equal(o, o2)  # and a second run gives the same bits


def test_prefill_scale_and_large_scores():
    # scores of a few hundred: the running maximum moves, rows become one-hot
    q, k, v = inputs(1, 600, 600, 8, 2, seed=5, mul=4.0)
    for scale in (0.5, 0.01):
        p = ops.Params(1, 8, 2, softmax_scale=scale)
        o, lse = ops.window_attn_prefill(p, q, k, v, 250, 8)
        w, z, tw, tz = attend(q[0], k[0], v[0], 0, 250, 8, scale=scale)
        # the scores' fp32 error grows with their size: scale 0.5 gives sum |q k| scale up to
        # ~128 x 16 x 0.5 ~ 1000, so P may be off by 1000 x DOT = 1.5e-2 where it is not 0 or 1
        slack = 1.6e-2 * v.abs().amax().double() * 2 if scale == 0.5 else 0.0
        close(o[0], w, tw + slack, f"scale {scale}")
        close(lse[0], z, tz, f"scale {scale} lse")


def test_prefill_rising_scores_rescale_the_sums():
    # key u scores higher than every earlier one: each tile raises the running maximum
    L = 1500
    q = torch.zeros(1, L, 4, 128, device="cuda")
    q[..., 0] = 8.0
    k = torch.zeros(1, 1, L, 128, device="cuda")
    k[..., 0] = (torch.arange(L, device="cuda") / 16).to(BF)[None, None]
    g = torch.Generator(device="cuda").manual_seed(9)
    v = randn(g, 1, 1, L, 128)
    q, k = q.to(BF), k.to(BF)
    o, lse = ops.window_attn_prefill(ops.Params(1, 4, 1), q, k, v, 700, 3)
    check_rows(o, lse, q, k, v, [L], [L], 700, 3, "rising")
    o, lse = ops.window_attn_prefill(ops.Params(1, 4, 1), q, -k, v, 700, 3)
    check_rows(o, lse, q, -k, v, [L], [L], 700, 3, "falling")


CHUNKS = [
    # Lq, Lmax, Hq, Hkv, window, n_sink, q_lens, kv_lens
    (7, 3000, 32, 2, 100000, 0, [7, 1, 3, 0], [3000, 1, 2000, 77]),
    (7, 3000, 16, 1, 200, 4, [7, 5], [3000, 130]),
    (130, 1000, 8, 2, 64, 65, [130, 17, 130], [1000, 999, 130]),
    (1, 20000, 4, 1, 5000, 64, [1, 1], [20000, 12345]),
    (300, 2500, 4, 4, 513, 1, [300, 299, 1], [2500, 300, 1]),
    (64, 40000, 32, 2, 40000, 0, [64], [39999]),
    (2, 64, 1, 1, 3, 0, [2, 2, 2, 2, 2], [64, 2, 63, 33, 5]),
]


@pytest.mark.parametrize("Lq,Lmax,Hq,Hkv,window,n_sink,ql,kl", CHUNKS)
def test_chunk_matches_reference_and_ignores_what_it_does_not_see(Lq, Lmax, Hq, Hkv, window, n_sink, ql, kl):
    B = len(ql)
    q, k, v = inputs(B, Lq, Lmax, Hq, Hkv, seed=Lmax + Lq)
    for b in range(B):
        q[b, ql[b]:] = NAN
        for x in (k, v):  # past the cache, and between the sinks and the first query's window
            x[b, :, kl[b]:] = NAN
            lo = kl[b] - ql[b] - window + 1
            if lo > n_sink:
                x[b, :, n_sink:lo] = NAN
                x[b, :, (n_sink + lo) // 2] = float("inf")
    p = ops.Params(B, Hq, Hkv)
    qt, kt = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (ql, kl))
    o = torch.full_like(q, 7.0)
    lse = torch.full((B, Hq, Lq), 7.0, device="cuda")
    ops.window_attn_chunk(p, q, k, v, window, n_sink, q_lens=qt, kv_lens=kt, out=o, lse=lse)
    check_rows(o, lse, q, k, v, ql, kl, window, n_sink, "chunk")
    for b in range(B):  # padding rows as they were
        assert (o[b, ql[b]:] == 7.0).all() and (lse[b, :, ql[b]:] == 7.0).all()


def test_chunk_clamps_lengths_on_the_gpu():
    q, k, v = inputs(3, 9, 50, 4, 2, seed=3)
    p = ops.Params(3, 4, 2)
    qt = torch.tensor([100, -5, 9], dtype=torch.int32, device="cuda")
    kt = torch.tensor([1000, 20, 4], dtype=torch.int32, device="cuda")
    o = torch.full_like(q, 7.0)
    _, lse = ops.window_attn_chunk(p, q, k, v, 30, 2, q_lens=qt, kv_lens=kt, out=o)
    check_rows(o, lse, q, k, v, [9, 0, 4], [50, 20, 4], 30, 2, "clamped")
    assert (o[1] == 7.0).all() and (o[2, 4:] == 7.0).all()


def test_chunk_rows_equal_those_of_a_prefill():
    q, k, v = inputs(1, 900, 900, 8, 1, seed=21)
    p = ops.Params(1, 8, 1)
    o, lse = ops.window_attn_prefill(p, q, k, v, 300, 5)
    oc, lc = ops.window_attn_chunk(p, q[:, 800:].contiguous(), k, v, 300, 5)
    w, z, tw, tz = attend(q[0], k[0], v[0], 0, 300, 5)
    close(oc[0], o[0, 800:].double(), 2 * tw[800:], "chunk against prefill")
    close(lc[0], lse[0, :, 800:].double(), 2 * tz[:, 800:], "chunk against prefill")


DECODE = [
    # Lmax, Hq, Hkv, window, n_sink, lens
    (1, 1, 1, 1, 0, [1]),
    (100, 16, 1, 16, 4, [100, 1, 16, 17, 20, 21, 64, 65]),
    (5000, 32, 2, 1000, 64, [5000, 64, 65, 1000, 1001, 1064, 1065, 4999]),
    (5000, 8, 8, 5000, 0, [5000, 3, 777]),
    (20000, 4, 1, 100000, 0, [20000]),
    (20000, 4, 2, 1, 0, [20000, 5]),
    (40000, 32, 2, 33333, 1, [40000, 39999, 12]),
    (128, 4, 2, 65, 60, [128, 127, 126, 125, 124, 64]),  # two runs: a segment more than the cache has blocks
    (64 * 9, 16, 1, 65, 62, [576, 128]),
    (300, 2, 1, 128, 128, [300, 255, 256, 257, 128, 129]),
    (70000, 16, 1, 70000, 0, [70000]),
    (2000, 16, 2, 500, 100, [2000 - 31 * i for i in range(64)]),
]


@pytest.mark.parametrize("Lmax,Hq,Hkv,window,n_sink,lens", DECODE)
def test_decode_matches_reference_and_ignores_what_it_does_not_see(Lmax, Hq, Hkv, window, n_sink, lens):
    B = len(lens)
    q, k, v = inputs(B, 1, Lmax, Hq, Hkv, seed=Lmax + B)
    for b in range(B):
        for x in (k, v):
            x[b, :, lens[b]:] = NAN
            if lens[b] - window > n_sink:
                x[b, :, n_sink:lens[b] - window] = NAN
    p = ops.Params(B, Hq, Hkv)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = ops.window_attn_decode(p, q[:, 0], k, v, lt, window, n_sink)
    check_rows(o[:, None], lse[..., None], q, k, v, [1] * B, lens, window, n_sink, "decode")
    o2, _ = ops.window_attn_decode(p, q[:, 0], k, v, lt, window, n_sink)
    assert torch.equal(o, o2)


# from one chunk to a cluster of 16 and past it, with sequences that end in its first and last chunks
@pytest.mark.parametrize("Lmax", [512, 513, 640, 1024, 2047, 3008, 3200])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (16, 1), (6, 3)])
def test_decode_joins_its_chunks(Lmax, Hq, Hkv):
    lens = [Lmax, 1, Lmax - 1, 129]
    q, k, v = inputs(len(lens), 1, Lmax, Hq, Hkv, seed=Lmax)
    p = ops.Params(len(lens), Hq, Hkv)
    lt = torch.tensor(lens, dtype=torch.int32, device="cuda")
    o, lse = ops.window_attn_decode(p, q[:, 0], k, v, lt, Lmax, 0)
    check_rows(o[:, None], lse[..., None], q, k, v, [1] * len(lens), lens, Lmax, 0, "decode")
    v[0, 0, Lmax - 1, 5] = NAN  # seen by sequence 0 alone, and by column 5 of its first group
    o2, lse2 = ops.window_attn_decode(p, q[:, 0], k, v, lt, Lmax, 0)
    nan = torch.zeros_like(o, dtype=torch.bool)
    nan[0, :Hq // Hkv, 5] = True
    assert torch.equal(o2.isnan(), nan) and torch.equal(lse, lse2) and torch.equal(o2[~nan], o[~nan])


def test_decode_empty_and_overlong_sequences():
    q, k, v = inputs(4, 1, 200, 8, 2, seed=2)
    lt = torch.tensor([0, -3, 1000, 5], dtype=torch.int32, device="cuda")
    o, lse = ops.window_attn_decode(ops.Params(4, 8, 2), q[:, 0], k, v, lt, 50, 2)
    assert (o[:2] == 0).all() and (lse[:2] == float("-inf")).all()
    check_rows(o[2:, None], lse[2:, :, None], q[2:], k[2:], v[2:], [1, 1], [200, 5], 50, 2, "clamped decode")


def test_decode_in_a_cache_whose_offsets_pass_32_bits():
    B, Lmax = 65, 262144  # 65 x 2 x 262144 x 128 elements: past 2^32
    p = ops.Params(B, 4, 2)
    g = torch.Generator(device="cuda").manual_seed(1)
    k = torch.zeros(B, 2, Lmax, 128, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    q = randn(g, B, 4, 128)
    lens = torch.full((B,), 100, dtype=torch.int32, device="cuda")
    lens[-1] = Lmax
    for x in (k, v):
        x[-1, :, -700:] = randn(g, 2, 700, 128)
        x[-1, :, :9] = randn(g, 2, 9, 128)
    o, lse = ops.window_attn_decode(p, q, k, v, lens, 700, 9)
    w, z, tw, tz = attend(q[-1:], torch.cat([k[-1, :, :9], k[-1, :, -700:]], 1),
                          torch.cat([v[-1, :, :9], v[-1, :, -700:]], 1), 708, 700, 9)
    close(o[-1:], w, tw, "o")
    close(lse[-1][:, None], z, tz, "lse")
    o, lse = ops.window_attn_chunk(p, q[:, None], k, v, 700, 9, kv_lens=lens)
    close(o[-1], w, tw, "chunk o")
    close(lse[-1], z, tz, "chunk lse")


BACKWARD = [
    # B, L, Hq, Hkv, window, n_sink, lens
    (1, 1, 1, 1, 1, 0, None),
    (1, 130, 16, 1, 16, 4, None),
    (2, 129, 8, 1, 64, 1, None),
    (1, 517, 32, 2, 128, 64, None),
    (1, 500, 4, 4, 1, 0, None),
    (1, 700, 8, 2, 10000, 0, None),
    (1, 300, 16, 1, 20, 500, None),
    (2, 1100, 4, 2, 256, 100, None),
    (1, 2100, 32, 2, 1000, 70, None),
    (1, 900, 2, 1, 2147483647, 3, None),
    (4, 400, 16, 2, 100, 4, [400, 1, 0, 257]),
    (3, 700, 4, 4, 64, 0, [128, 700, 129]),
]


@pytest.mark.parametrize("B,L,Hq,Hkv,window,n_sink,lens", BACKWARD)
def test_backward_matches_reference(B, L, Hq, Hkv, window, n_sink, lens):
    q, k, v = inputs(B, L, L, Hq, Hkv, seed=L + 3 * window % 1000)
    do = randn(torch.Generator(device="cuda").manual_seed(L), B, L, Hq, 128)
    p = ops.Params(B, Hq, Hkv)
    n = lens or [L] * B
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    for b in range(B):  # what lies in the padding does not matter
        for x in (q, do):
            x[b, n[b]:] = NAN
        for x in (k, v):
            x[b, :, n[b]:] = NAN
    o = torch.full_like(q, NAN)
    lse = torch.full((B, Hq, L), NAN, device="cuda")
    ops.window_attn_chunk(p, q, k, v, window, n_sink, q_lens=lt, kv_lens=lt, out=o, lse=lse)
    out = [torch.full_like(x, 7.0) for x in (q, k, v)]
    got = ops.window_attn_backward(p, q, k, v, o, lse, do, window, n_sink, lens=lt, dq=out[0], dk=out[1], dv=out[2])
    for b in range(B):
        m = n[b]
        if m:
            ref, tol = attend_backward(q[b, :m], k[b, :, :m], v[b, :, :m], o[b, :m], lse[b, :, :m], do[b, :m],
                                       window, n_sink)
            close(got[0][b, :m], ref[0], tol[0], f"dq[{b}]")
            close(got[1][b, :, :m], ref[1], tol[1], f"dk[{b}]")
            close(got[2][b, :, :m], ref[2], tol[2], f"dv[{b}]")
        assert (got[0][b, m:] == 7.0).all() and (got[1][b, :, m:] == 7.0).all() and (got[2][b, :, m:] == 7.0).all()
    again = ops.window_attn_backward(p, q, k, v, o, lse, do, window, n_sink, lens=lt, dq=out[0].clone(),
                                     dk=out[1].clone(), dv=out[2].clone())
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # deterministic


def test_backward_against_differences():
    # d(sum O dO) along a random direction, by central differences of the fp64 forward
    B, L, Hq, Hkv, W, ns = 1, 200, 4, 2, 60, 3
    q, k, v = inputs(B, L, L, Hq, Hkv, seed=77)
    g = torch.Generator(device="cuda").manual_seed(78)
    do = randn(g, B, L, Hq, 128)
    p = ops.Params(B, Hq, Hkv)
    o, lse = ops.window_attn_prefill(p, q, k, v, W, ns)
    grads = ops.window_attn_backward(p, q, k, v, o, lse, do, W, ns)
    _, tol = attend_backward(q[0], k[0], v[0], o[0], lse[0], do[0], W, ns)
    # the kernel's D uses the rounded O: D is off by at most 2^-8 sum |dO| (|o| + sum P |v|), which
    # shifts dS by P times that; P sums to 1, so dq by scale max|k| and dk by scale sum P |q| of it
    x = [t[0].double() for t in (q, k, v)]

    def loss(a, b, c):
        return float((attend(a, b, c, 0, W, ns)[0] * do[0].double()).sum())
    dd = 2.0 ** -7 * (do.abs().double().sum(-1).amax() * v.abs().double().amax())
    slack = [128 ** -0.5 * dd * k.abs().double().amax(), 128 ** -0.5 * dd * q.abs().double().amax() * Hq // Hkv, 0.0]
    for i, name in enumerate(("dq", "dk", "dv")):
        u = torch.randn(x[i].shape, generator=g, device="cuda", dtype=torch.float64)
        u[torch.rand(u.shape[:-1], generator=g, device="cuda") < 0.9] = 0  # a few rows
        h = 1e-5
        lo, hi = ([t - h * u if j == i else t for j, t in enumerate(x)],
                  [t + h * u if j == i else t for j, t in enumerate(x)])
        want = (loss(*hi) - loss(*lo)) / (2 * h)
        gr = grads[i][0].double()
        bound = float(((tol[i] + slack[i]) * u.abs()).sum())
        assert abs(float((gr * u).sum()) - want) <= bound, name
        # and the bound is not vacuous for the direction of the gradient itself
        assert float((gr * gr).sum()) > 0


def test_calls_on_two_streams_and_in_a_graph():
    q, k, v = inputs(2, 300, 300, 8, 2, seed=31)
    p = ops.Params(2, 8, 2)
    lens = torch.tensor([300, 123], dtype=torch.int32, device="cuda")
    want = ops.window_attn_prefill(p, q, k, v, 100, 4)[0]
    wantd = ops.window_attn_decode(p, q[:, 0].contiguous(), k, v, lens, 100, 4)[0]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    res = []
    for s in (s1, s2):
        with torch.cuda.stream(s):
            for _ in range(3):
                res.append((ops.window_attn_prefill(p, q, k, v, 100, 4)[0],
                            ops.window_attn_decode(p, q[:, 0].contiguous(), k, v, lens, 100, 4)[0]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, wantd) for a, b in res)
    # captured and replayed on new inputs in the same buffers
    do = torch.randn_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = ops.window_attn_prefill(p, q, k, v, 100, 4)
        gr = ops.window_attn_backward(p, q, k, v, o, lse, do, 100, 4)
        od, _ = ops.window_attn_decode(p, q[:, 0].contiguous(), k, v, lens, 100, 4)
    q2, k2, v2 = inputs(2, 300, 300, 8, 2, seed=32)
    q.copy_(q2), k.copy_(k2), v.copy_(v2)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    o2, lse2 = ops.window_attn_prefill(p, q, k, v, 100, 4)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(a, b) for a, b in zip(gr, ops.window_attn_backward(p, q, k, v, o, lse, do, 100, 4)))
    assert torch.equal(od, ops.window_attn_decode(p, q[:, 0].contiguous(), k, v, lens, 100, 4)[0])


def test_binding_refusals():
    q, k, v = inputs(1, 8, 16, 4, 2, seed=1)
    p = ops.Params(1, 4, 2)
    lens = torch.tensor([8], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        ops.window_attn_chunk(p, q.transpose(1, 2).contiguous().transpose(1, 2), k, v, 4)
    with pytest.raises(ValueError, match="bfloat16"):
        ops.window_attn_chunk(p, q.half(), k, v, 4)
    with pytest.raises(ValueError, match="tokens"):
        ops.window_attn_prefill(p, q, k, v, 4)
    with pytest.raises(ValueError, match="int32"):
        ops.window_attn_decode(p, q[:, 0].contiguous(), k, v, lens.long(), 4)
    for w, s in ((0, 0), (-1, 0), (4, -1)):
        with pytest.raises(_lib.InfLLMv2Error, match="invalid argument"):
            ops.window_attn_chunk(p, q, k, v, w, s)
        with pytest.raises(_lib.InfLLMv2Error, match="invalid argument"):
            ops.window_attn_decode(p, q[:, 0].contiguous(), k, v, lens, w, s)
