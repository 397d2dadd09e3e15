"""Per-head norm with rotation (forward, backward, table) against the fp64 reference, and the
whole layer path: projection rows -> norm and rotation -> caches -> attention -> gradients."""
import pytest
import torch

from window_ref import attend, attend_backward, close, norm_rope, norm_rope_backward
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
    assert ops.device_error(clear=True) == 0


def randn(g, *shape, mul=1.0, add=0.0):
    return (mul * torch.randn(*shape, generator=g, device="cuda") + add).to(BF)


def inv_freq(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).float().cuda()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def projection(B, L, Hq, Hkv, seed, pad=0):
    """Views q, k, v of packed rows (with `pad` unused elements behind each)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    H = Hq + 2 * Hkv
    rows = randn(g, B, L, H * 128 + pad, mul=2.0)
    x = rows[..., :H * 128].unflatten(-1, (H, 128)) if pad else rows.view(B, L, H, 128)
    return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]


def weights(kind, seed):
    if kind is None:
        return None, None
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = [randn(g, 128, mul=0.3, add=1.0) for _ in range(2)]
    return [x.to(torch.float32 if kind == "fp32" else BF) for x in w]


@pytest.mark.parametrize("rot,n,scale", [(16, 1, 1.0), (128, 262144, 1.0), (96, 1000, 1.25)])
def test_rope_table(rot, n, scale):
    f = inv_freq(rot)
    t = ops.rope_table(ops.Params(1, 1, 1), f, n, scale)
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * f.double()
    want = scale * torch.cat([ang.cos(), ang.sin()], 1)
    # one rounding of a value of at most `scale`; the fp64 angle is off by at most 2^-53 x 262144
    close(t, want, 2.0 ** -24 * scale + 1e-9, "table")


CASES = [
    # B, L, Hq, Hkv, rot, interleaved, weights, pad
    (1, 1, 1, 1, 128, False, "bf16", 0),
    (3, 1, 32, 2, 128, False, "bf16", 0),
    (2, 37, 16, 2, 64, True, "fp32", 0),
    (1, 1000, 8, 1, 128, False, None, 8),
    (2, 515, 4, 4, 16, False, "fp32", 64),
    (1, 333, 32, 8, 96, True, "bf16", 0),
    (2, 129, 2, 1, 48, False, "bf16", 24),
    (1, 20000, 4, 2, 128, True, "bf16", 0),
]


@pytest.mark.parametrize("B,L,Hq,Hkv,rot,interleaved,wk,pad", CASES)
def test_forward_and_backward_fresh(B, L, Hq, Hkv, rot, interleaved, wk, pad):
    p = ops.Params(B, Hq, Hkv)
    q, k, v = projection(B, L, Hq, Hkv, seed=L, pad=pad)
    qw, kw = weights(wk, L)
    table = ops.rope_table(p, inv_freq(rot), L + 5)
    kwargs = dict(q_weight=qw, k_weight=kw, eps=1e-5, interleaved=interleaved)
    qo, ko, vo = ops.qk_norm_rope(p, q, k, v, table, **kwargs)
    g = torch.Generator(device="cuda").manual_seed(L + 1)
    dq, dk, dv = randn(g, B, L, Hq, 128), randn(g, B, Hkv, L, 128), randn(g, B, Hkv, L, 128)
    gq, gk, gv, gqw, gkw = ops.qk_norm_rope_backward(p, q, k, dq, dk, dv, table, **kwargs)
    dws = [[0, 0], [0, 0]]
    for b in range(B):
        for got, x, w, name in ((qo[b], q[b], qw, "q"), (ko[b].transpose(0, 1), k[b], kw, "k")):
            want, tol = norm_rope(x, w, 1e-5, table[:L], interleaved)
            close(got, want, tol, name)
        for i, (got, x, w, d) in enumerate(((gq[b], q[b], qw, dq[b]), (gk[b], k[b], kw, dk[b].transpose(0, 1)))):
            dx, tol, dw, tw = norm_rope_backward(x, w, 1e-5, table[:L], interleaved, d)
            close(got, dx, tol, f"d{'qk'[i]}")
            dws[i][0], dws[i][1] = dws[i][0] + dw, dws[i][1] + tw
    assert torch.equal(vo, v.transpose(1, 2)) and torch.equal(gv, dv.transpose(1, 2))
    if wk is None:
        assert gqw is None and gkw is None
    else:
        close(gqw, dws[0][0], dws[0][1], "d_qw")
        close(gkw, dws[1][0], dws[1][1], "d_kw")
        again = ops.qk_norm_rope_backward(p, q, k, dq, dk, dv, table, **kwargs)
        assert torch.equal(gqw, again[3]) and torch.equal(gkw, again[4])  # a fixed order


def test_chunks_into_caches_and_lengths():
    B, L, Hq, Hkv, Lmax = 5, 40, 8, 2, 300
    p = ops.Params(B, Hq, Hkv)
    q, k, v = projection(B, L, Hq, Hkv, seed=4)
    qw, kw = weights("fp32", 4)
    table = ops.rope_table(p, inv_freq(64), Lmax)
    n = [40, 0, 17, 1, 40]
    starts, q_lens = i32(0, 300, 283, 7, 260), i32(400, -1, 17, 1, 40)
    lens_out = i32(-9, -9, -9, -9, -9)
    for b in range(B):
        for x in (q, k, v):
            x[b, n[b]:] = NAN  # padding is not read
    kc, vc = torch.full((B, Hkv, Lmax, 128), 7.0, dtype=BF, device="cuda"), \
        torch.full((B, Hkv, Lmax, 128), 7.0, dtype=BF, device="cuda")
    qo = torch.full((B, L, Hq, 128), 7.0, dtype=BF, device="cuda")
    got = ops.qk_norm_rope(p, q, k, v, table, qw, kw, starts=starts, q_lens=q_lens, k_cache=kc, v_cache=vc, q_out=qo,
                           lens_out=lens_out)
    assert got[0] is qo and got[1] is kc and got[2] is vc
    assert lens_out.tolist() == [40, 300, 300, 8, 300]
    for b in range(B):
        m, t0 = n[b], int(starts[b])
        rows = torch.ones(Lmax, dtype=torch.bool, device="cuda")
        if m:
            want, tol = norm_rope(q[b, :m], qw, 1e-6, table[t0:t0 + m], False)
            close(qo[b, :m], want, tol, "q")
            want, tol = norm_rope(k[b, :m], kw, 1e-6, table[t0:t0 + m], False)
            close(kc[b, :, t0:t0 + m].transpose(0, 1), want, tol, "k")
            assert torch.equal(vc[b, :, t0:t0 + m].transpose(0, 1), v[b, :m])
            rows[t0:t0 + m] = False
        assert (qo[b, m:] == 7.0).all() and (kc[b, :, rows] == 7.0).all() and (vc[b, :, rows] == 7.0).all()


def test_rows_past_the_cache_or_the_table_are_refused_on_the_gpu():
    B, L, Lmax = 4, 3, 20
    p = ops.Params(B, 2, 1)
    q, k, v = projection(B, L, 2, 1, seed=6)
    starts = i32(17, 18, -1, 2147483647)
    table = ops.rope_table(p, inv_freq(128), 64)
    kc = torch.full((B, 1, Lmax, 128), 7.0, dtype=BF, device="cuda")
    vc, qo, lens_out = kc.clone(), torch.full((B, L, 2, 128), 7.0, dtype=BF, device="cuda"), i32(0, 0, 0, 0)
    ops.qk_norm_rope(p, q, k, v, table, starts=starts, k_cache=kc, v_cache=vc, q_out=qo, lens_out=lens_out)
    assert ops.device_error(clear=True) == _lib.DEVERR_CACHE_FULL
    assert lens_out.tolist() == [20, 18, -1, 2147483647]
    assert (kc[0, :, :17] == 7).all() and not (kc[0, :, 17:] == 7).any()
    for x in (kc, vc, qo):
        assert (x[1:] == 7.0).all()
    # the table is too short (fresh outputs): the sequence is left alone
    ops.qk_norm_rope(p, q, k, v, ops.rope_table(p, inv_freq(128), 20), starts=starts, q_out=qo)
    assert ops.device_error(clear=True) == _lib.DEVERR_CACHE_FULL
    assert (qo[1:] == 7.0).all()
    g = torch.Generator(device="cuda").manual_seed(1)
    dq, dk = randn(g, B, L, 2, 128), randn(g, B, 1, L, 128)
    w = torch.ones(128, device="cuda")
    out = torch.full((B, L, 4, 128), 7.0, dtype=BF, device="cuda")
    r = ops.qk_norm_rope_backward(p, q, k, dq, dk, dk, table[:20].contiguous(), w, w, starts=starts, out=out)
    assert ops.device_error(clear=True) == _lib.DEVERR_CACHE_FULL
    assert (out[1:] == 7.0).all() and torch.isfinite(out[0]).all()
    one = ops.Params(1, 2, 1)
    r1 = ops.qk_norm_rope_backward(one, q[:1], k[:1], dq[:1], dk[:1], dk[:1], table, w, w, starts=starts[:1])
    close(r[3], r1[3].double(), 1e-5 * 6 * 128 ** 0.5 * r1[3].abs().double().amax(), "d_qw of the sequence that fits")


def test_zero_rows_and_backward_padding():
    p = ops.Params(2, 4, 1)
    q, k, v = projection(2, 50, 4, 1, seed=8)
    q[:, 3] = 0  # a zero row: y = 0, and its gradient is finite
    table = ops.rope_table(p, inv_freq(32), 50)
    qo, _, _ = ops.qk_norm_rope(p, q, k, v, table)
    assert (qo[:, 3] == 0).all()
    g = torch.Generator(device="cuda").manual_seed(1)
    dq, dk = randn(g, 2, 50, 4, 128), randn(g, 2, 1, 50, 128)
    w = torch.ones(128, device="cuda")
    lens = i32(50, 21)
    for x in (dq, dk.transpose(1, 2)):
        x[1, 21:] = NAN
    out = torch.full((2, 50, 6, 128), 7.0, dtype=BF, device="cuda")
    r = ops.qk_norm_rope_backward(p, q, k, dq, dk, dk, table, w, w, q_lens=lens, out=out)
    assert torch.isfinite(out[0]).all() and torch.isfinite(out[1, :21]).all() and (out[1, 21:] == 7.0).all()
    dw = tw = 0
    for b, n in ((0, 50), (1, 21)):
        dx, tol, d, t = norm_rope_backward(q[b, :n], w, 1e-6, table[:n], False, dq[b, :n])
        close(r[0][b, :n], dx, tol, "dq")
        dw, tw = dw + d, tw + t
    close(r[3], dw, tw, "d_qw")


# several chunks of query and of key and value heads, with ragged ends, padding and an empty sequence
@pytest.mark.parametrize("L,Hq,Hkv", [(1201, 10, 10), (900, 16, 16), (2050, 5, 5), (1400, 36, 9), (701, 14, 7)])
def test_backward_over_chunks_of_heads(L, Hq, Hkv):
    p = ops.Params(3, Hq, Hkv)
    q, k, v = projection(3, L, Hq, Hkv, seed=L)
    n, t0 = [L, L - 77, 0], [0, 40, 3]
    for b in range(3):
        q[b, n[b]:], k[b, n[b]:] = NAN, NAN
    qw, kw = weights("fp32", L)
    table = ops.rope_table(p, inv_freq(96), L)
    g = torch.Generator(device="cuda").manual_seed(L)
    dq, dk, dv = (randn(g, *x) for x in ((3, L, Hq, 128), (3, Hkv, L, 128), (3, Hkv, L, 128)))
    out = torch.full((3, L, Hq + 2 * Hkv, 128), 7., dtype=BF, device="cuda")
    r = ops.qk_norm_rope_backward(p, q, k, dq, dk, dv, table, qw, kw, starts=i32(*t0), q_lens=i32(*n), out=out)
    want = {3: [0., 0.], 4: [0., 0.]}
    for b in range(2):
        m, tab = n[b], table[t0[b]:t0[b] + n[b]]
        for i, x, w, d in ((0, q, qw, dq[b, :m]), (1, k, kw, dk[b, :, :m].transpose(0, 1))):
            dx, tol, dw, tw = norm_rope_backward(x[b, :m], w, 1e-6, tab, False, d)
            close(r[i][b, :m], dx, tol, "dx")
            want[3 + i] = [want[3 + i][0] + dw, want[3 + i][1] + tw]
        assert torch.equal(r[2][b, :m], dv[b, :, :m].transpose(0, 1))
        assert (out[b, m:] == 7).all()
    assert (out[2] == 7).all()
    for i in (3, 4):
        close(r[i], *want[i], "dw")
    r2 = ops.qk_norm_rope_backward(p, q, k, dq, dk, dv, table, qw, kw, starts=i32(*t0), q_lens=i32(*n))
    assert torch.equal(r[3], r2[3]) and torch.equal(r[4], r2[4])


def test_backward_against_differences():
    p = ops.Params(1, 2, 1)
    q, k, v = projection(1, 9, 2, 1, seed=14)
    qw, kw = weights("fp32", 3)
    table = ops.rope_table(p, inv_freq(64), 9)
    g = torch.Generator(device="cuda").manual_seed(2)
    dq, dk = randn(g, 1, 9, 2, 128), randn(g, 1, 1, 9, 128)
    r = ops.qk_norm_rope_backward(p, q, k, dq, dk, dk, table, qw, kw, interleaved=True)
    dx, tol, dw, tw = norm_rope_backward(q[0], qw, 1e-6, table, True, dq[0])

    def loss(x, w):
        return float((norm_rope(x, w, 1e-6, table, True)[0] * dq[0].double()).sum())
    x, w, h = q[0].double(), qw.double(), 1e-6
    u = torch.randn(x.shape, generator=g, device="cuda", dtype=torch.float64)
    want = (loss(x + h * u, w) - loss(x - h * u, w)) / (2 * h)
    assert abs(float((r[0][0].double() * u).sum()) - want) <= float((tol * u.abs()).sum()) + 1e-5 * abs(want)
    u = torch.randn(128, generator=g, device="cuda", dtype=torch.float64)
    want = (loss(x, w + h * u) - loss(x, w - h * u)) / (2 * h)
    assert abs(float((r[3].double() * u).sum()) - want) <= float((tw * u.abs()).sum()) + 1e-5 * abs(want)


def test_binding_refusals():
    p = ops.Params(2, 4, 1)
    q, k, v = projection(2, 6, 4, 1, seed=1)
    table = ops.rope_table(p, inv_freq(128), 6)
    w = torch.ones(128, device="cuda")
    bad = [dict(q=q.transpose(2, 3)), dict(q=q[:, ::2]), dict(k=k.float()), dict(q=q[:1]),
           dict(table=table.double()), dict(q_weight=w, k_weight=w.to(BF)), dict(q_weight=w.half()),
           dict(q_weight=w[:64]), dict(starts=i32(0)), dict(starts=i32(0, 0).long()),
           dict(k_cache=torch.zeros(2, 1, 9, 128, dtype=BF, device="cuda"))]
    for b in bad:
        kw = {**dict(q=q, k=k, v=v, table=table), **b}
        with pytest.raises(ValueError):
            ops.qk_norm_rope(p, kw.pop("q"), kw.pop("k"), kw.pop("v"), kw.pop("table"), **kw)
    s = i32(0, 0)
    for b in (dict(eps=0.0), dict(eps=NAN), dict(starts=s, lens_out=s)):
        with pytest.raises(_lib.InfLLMv2Error, match="invalid argument"):
            ops.qk_norm_rope(p, q, k, v, table, **b)
    with pytest.raises(_lib.InfLLMv2Error, match="invalid argument"):
        ops.qk_norm_rope(p, q, k, v, ops.rope_table(p, inv_freq(128), 6)[:, :120].contiguous())
    with pytest.raises(ValueError, match="one stride"):
        ops.qk_norm_rope(p, q[:, :1].expand(2, 6, 4, 128), k, v, table)  # every token one row
    with pytest.raises(_lib.InfLLMv2Error, match="invalid argument"):
        ops.rope_table(p, torch.ones(7, device="cuda"), 6)


def test_layer_path_prefill_decode_and_training():
    """Projection rows through the operators as a model runs them: a prompt in two chunks, decode
    steps of a window layer and of a sparse layer, and a training step; every stage against the
    reference of that stage on the stage's own inputs."""
    B, Hq, Hkv, Lmax, W, ns = 2, 16, 1, 600, 128, 16
    p = ops.Params(B, Hq, Hkv, topk=4)
    qw, kw = weights("bf16", 1)
    table = ops.rope_table(p, inv_freq(128), Lmax)
    kc, vc = (torch.full((B, Hkv, Lmax, 128), NAN, dtype=BF, device="cuda") for _ in range(2))
    lens = i32(0, 0)
    for n in ([300, 170], [201, 64]):
        L = max(n)
        q, k, v = projection(B, L, Hq, Hkv, seed=L)
        q_lens, new = i32(*n), torch.empty_like(lens)
        qo, _, _ = ops.qk_norm_rope(p, q, k, v, table, qw, kw, starts=lens, q_lens=q_lens, k_cache=kc, v_cache=vc,
                                    lens_out=new)
        o, lse = ops.window_attn_chunk(p, qo, kc, vc, W, ns, q_lens=q_lens, kv_lens=new)
        for b in range(B):
            t0 = int(lens[b])
            want, tol = norm_rope(k[b, :n[b]], kw, 1e-6, table[t0:t0 + n[b]], False)
            close(kc[b, :, t0:t0 + n[b]].transpose(0, 1), want, tol, "cached keys")
            w, z, tw, tz = attend(qo[b, :n[b]], kc[b, :, :t0 + n[b]], vc[b, :, :t0 + n[b]], t0, W, ns)
            close(o[b, :n[b]], w, tw, "chunk")
        lens = new
    assert lens.tolist() == [501, 234]
    # decode: one projected token per sequence, appended, then attended to
    for step in range(3):
        q, k, v = projection(B, 1, Hq, Hkv, seed=900 + step)
        new = torch.empty_like(lens)
        kc2, vc2 = kc.clone(), vc.clone()
        qo, _, _ = ops.qk_norm_rope(p, q, k, v, table, qw, kw, starts=lens, k_cache=kc, v_cache=vc, lens_out=new)
        o, _ = ops.window_attn_decode(p, qo[:, 0], kc, vc, new, W, ns)
        for b in range(B):
            n = int(new[b])
            w, z, tw, tz = attend(qo[b], kc[b, :, :n], vc[b, :, :n], n - 1, W, ns)
            close(o[b][None], w, tw, "decode")
        # the same token through the sparse layer's step: fresh rows, appended by decode_step
        qf, kf, vf = ops.qk_norm_rope(p, q, k, v, table, qw, kw, starts=lens)
        assert torch.equal(qf, qo)
        sem = ops.compress_keys(p, kc2, lens=lens)
        _, _, _, after = ops.decode_step(p, qf[:, 0], kc2, vc2, sem, lens, k_new=kf[:, :, 0], v_new=vf[:, :, 0])
        assert torch.equal(after, new)
        for b in range(B):
            n = int(new[b])
            assert torch.equal(kc2[b, :, :n], kc[b, :, :n]) and torch.equal(vc2[b, :, :n], vc[b, :, :n])
        lens = new
    # training: forward and backward of one layer
    L = 260
    q, k, v = projection(B, L, Hq, Hkv, seed=40)
    do = randn(torch.Generator(device="cuda").manual_seed(41), B, L, Hq, 128)
    qo, ko, vo = ops.qk_norm_rope(p, q, k, v, table, qw, kw)
    o, lse = ops.window_attn_prefill(p, qo, ko, vo, W, ns)
    dq, dk, dv = ops.window_attn_backward(p, qo, ko, vo, o, lse, do, W, ns)
    gq, gk, gv, gqw, gkw = ops.qk_norm_rope_backward(p, q, k, dq, dk, dv, table, qw, kw)
    dwk = twk = 0
    for b in range(B):
        ref, tol = attend_backward(qo[b], ko[b], vo[b], o[b], lse[b], do[b], W, ns)
        for got, r, t in zip((dq[b], dk[b], dv[b]), ref, tol):
            close(got, r, t, "attention gradients")
        dx, tol, dw, tw = norm_rope_backward(k[b], kw, 1e-6, table[:L], False, dk[b].transpose(0, 1))
        close(gk[b], dx, tol, "dk of the projection")
        dwk, twk = dwk + dw, twk + tw
    close(gkw, dwk, twk, "d_kw")
