"""Plain fp64 references of the window attention and of the per-head norm with rotation,
with elementwise error bounds for the kernels (plain torch, no code of the library).

Bounds.  eps(bf16) / 2 = 2^-8 is the relative error of one rounding to bf16.
 * O: the probabilities are rounded to bf16 before the product with V (2^-8 sum P |v|), the
   result once more (2^-8 |o|); the fp32 scores and sums add less than 2e-4 sum P |v|: a
   score is a 128-term fp32 dot product, off by at most 128 x 2^-23 of sum |q k| scale (a few
   1e-5 of scores of size ~10).
 * lse: the same fp32 dot products, plus the hardware exp2 / log2 (2^-20 of 1 + |lse|).
 * dV as O; dS = P (dP - D) is rounded once (2^-8 |dS|) after fp32 dot products dP and D (each
   128 x 2^-23 = 2^-16 of its absolute terms) with the P error above; dq and dK are its
   products, rounded once.
 * norm and rotation: one rounding of the result; fp32 arithmetic in between, a handful of
   operations of 2^-24 and a 128-term sum: 1e-5 of the terms.
"""
import math

import torch

H8 = 2.0 ** -8
F32 = 2.0e-4   # fp32 part of P's relative error (scores up to a few tens)
DOT = 128 * 2.0 ** -23


def visible(t, u, window, n_sink):
    return (u[None, :] <= t[:, None]) & ((u[None, :] > t[:, None] - window) | (u[None, :] < n_sink))


def attend(q, k, v, first, window, n_sink, scale=None):
    """q [R, Hq, d] at positions first.., k, v [Hkv, N, d] -> o, lse [Hq, R] and their bounds."""
    R, Hq, d = q.shape
    Hkv, N, _ = k.shape
    scale = scale or 1 / math.sqrt(d)
    q, k, v = q.double(), k.double(), v.double()
    ok = visible(torch.arange(first, first + R, device=q.device), torch.arange(N, device=q.device), window, n_sink)
    o, lse, to, tl = [], [], [], []
    for h in range(Hq):
        g = h // (Hq // Hkv)
        seen = ok.any(0)
        kk = torch.where(seen[:, None], k[g], torch.zeros((), dtype=torch.float64, device=q.device))
        vv = torch.where(seen[:, None], v[g], torch.zeros((), dtype=torch.float64, device=q.device))
        x = (q[:, h] @ kk.T * scale).masked_fill(~ok, -math.inf)
        z = torch.logsumexp(x, -1)
        pr = torch.exp(x - z[:, None])
        oh = pr @ vv
        a = pr @ vv.abs()
        xa = (q[:, h].abs() @ kk.abs().T * abs(scale)).masked_fill(~ok, 0).amax(-1)
        o.append(oh)
        lse.append(z)
        to.append(H8 * (oh.abs() + a) * (1 + H8) + F32 * a)
        tl.append(DOT * xa + 2.0 ** -20 * (1 + z.abs()))
    return torch.stack(o, 1), torch.stack(lse), torch.stack(to, 1), torch.stack(tl)


def attend_backward(q, k, v, o, lse, do, window, n_sink, scale=None):
    """Gradients over one fresh sequence and their bounds: (dq, dk, dv), (tq, tk, tv)."""
    R, Hq, d = q.shape
    Hkv = k.shape[0]
    G = Hq // Hkv
    scale = scale or 1 / math.sqrt(d)
    q, k, v, o, lse, do = (x.double() for x in (q, k, v, o, lse, do))
    i = torch.arange(R, device=q.device)
    ok = visible(i, i, window, n_sink)
    dq, tq = torch.zeros_like(q), torch.zeros_like(q)
    dk, dv, tk, tv = (torch.zeros_like(k) for _ in range(4))
    ak, av = torch.zeros_like(k), torch.zeros_like(k)
    for h in range(Hq):
        g = h // G
        pr = torch.exp(q[:, h] @ k[g].T * scale - lse[h][:, None]).masked_fill(~ok, 0)
        D = (do[:, h] * o[:, h]).sum(-1, keepdim=True)
        ds = pr * (do[:, h] @ v[g].T - D)
        e = H8 * ds.abs() + F32 * ds.abs() + 1.01 * pr * DOT * (
            do[:, h].abs() @ v[g].abs().T + (do[:, h].abs() * o[:, h].abs()).sum(-1, keepdim=True))
        dq[:, h] = scale * ds @ k[g]
        tq[:, h] = H8 * dq[:, h].abs() + 1.01 * scale * e @ k[g].abs()
        dk[g] += scale * ds.T @ q[:, h]
        ak[g] += 1.01 * scale * e.T @ q[:, h].abs()
        dv[g] += pr.T @ do[:, h]
        av[g] += (1.01 * H8 + F32) * pr.T @ do[:, h].abs()
    tk, tv = H8 * dk.abs() + ak, H8 * dv.abs() + av
    return (dq, dk, dv), (tq, tk, tv)


def rotate(y, table, interleaved, sign=1.0):
    """y [R, ..., d] by the rows of table [R, rot] (cos, then sin)."""
    rot = table.shape[1]
    sh = [table.shape[0]] + [1] * (y.dim() - 2) + [rot // 2]
    c, s = table[:, :rot // 2].double().reshape(sh), sign * table[:, rot // 2:].double().reshape(sh)
    i = torch.arange(rot // 2, device=y.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    out = y.clone()
    out[..., a] = y[..., a] * c - y[..., b] * s
    out[..., b] = y[..., a] * s + y[..., b] * c
    return out


def norm_rope(x, w, eps, table, interleaved):
    """x [R, H, d] -> y and its bound."""
    x = x.double()
    y = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.double()
    out = rotate(y, table, interleaved)
    return out, H8 * out.abs() + 1e-5 * y.abs().amax(-1, keepdim=True)


def norm_rope_backward(x, w, eps, table, interleaved, dy):
    """x, dy [R, H, d] -> dx, its bound, dw [d], its bound."""
    x, g = x.double(), rotate(dy.double(), table, interleaved, -1.0)
    r = 1 / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps)
    gw = g if w is None else g * w.double()
    dx = r * gw - x * r ** 3 * (gw * x).mean(-1, keepdim=True)
    terms = (r * gw).abs() + (x * r ** 3).abs() * (gw * x).abs().mean(-1, keepdim=True)
    dw = (g * x * r).sum((0, 1))
    # g itself is a rotation in fp32: its error goes by the pair's size, so by the row's
    gmax = g.abs().amax(-1, keepdim=True)
    wmax = 1.0 if w is None else w.double().abs().amax()
    tdx = H8 * dx.abs() + 1e-5 * (terms + r * gmax * wmax * 2)
    tdw = 1e-5 * ((g.abs() + gmax) * x.abs() * r).sum((0, 1))
    return dx, tdx, dw, tdw


def close(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = (got - want).abs() - tol
    assert float(bad.max()) <= 0, f"{what}: {int((bad > 0).sum())} of {bad.numel()} values past their bound, by {float(bad.max()):.3g}"
