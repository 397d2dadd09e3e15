"""What the norm-and-rotation pass and the sliding-window attention are measured on.

Two operators around the block-sparse attention:

* ``qk_norm_rope``: per-head RMS norm of q and k and their position rotation in one pass, from the
  projection's layout into the attention's (q token-major, k and v head-major, fresh or in the caches),
  and its backward;
* ``window_attn``: attention over the last ``window`` keys and the first ``n_sink`` keys, for a fresh
  prefill, a ragged chunk against caches, decode, and the backward.

``run`` computes either the plain form (elementary torch operations in fp32, rounded once) or, with
``own`` set, the framework's calls.  ``exact`` is the definition in fp64.
"""
import math

import torch

own = False

D = 128


# ----------------------------------------------------------------------------- cases
def _rope(name, kind, B, L, Hq, Hkv, rot=D, interleaved=False, Lmax=0, ragged=False, wtype="bf16"):
    return {"name": name, "op": "rope", "kind": kind, "B": B, "L": L, "Hq": Hq, "Hkv": Hkv, "rot": rot,
            "interleaved": interleaved, "Lmax": Lmax, "ragged": ragged, "wtype": wtype}


def _win(name, kind, B, L, Hq, Hkv, window, n_sink, Lmax=0, ragged=False):
    return {"name": name, "op": "win", "kind": kind, "B": B, "L": L, "Hq": Hq, "Hkv": Hkv, "window": window,
            "n_sink": n_sink, "Lmax": Lmax, "ragged": ragged}


def listed():
    return [
        # the new token of one sequence before a decode step: launch latency
        _rope("rope_decode_b1", "decode", 1, 1, 32, 2, Lmax=32768),
        # a ragged batch of chunks written into caches, half of each head rotated, neighbouring pairs
        _rope("rope_chunk_ragged", "chunk", 5, 1000, 32, 4, rot=64, interleaved=True, Lmax=8192, ragged=True,
              wtype="fp32"),
        # the whole projection of a 128K prompt
        _rope("rope_prefill_128k", "fresh", 1, 131072, 32, 2),
        # a training step's sequence, odd length
        _rope("rope_backward_16k", "backward", 2, 8191, 32, 2),
        # a short prompt through one window layer
        _win("win_prefill_2k", "prefill", 1, 2048, 8, 1, 512, 64),
        # plain causal attention of a batch (window longer than the sequence), four heads a group
        _win("win_prefill_dense_8k", "prefill", 2, 8191, 32, 8, 8192, 0),
        # a 128K prompt through one window layer
        _win("win_prefill_128k", "prefill", 1, 131072, 32, 2, 4096, 64),
        # a few drafted tokens per sequence checked against long caches, every key visible
        _win("win_chunk_verify", "chunk", 4, 7, 32, 2, 131072, 0, Lmax=65536, ragged=True),
        # one token of a small batch, window layer: latency
        _win("win_decode_b8_32k", "decode", 8, 1, 32, 2, 4096, 64, Lmax=32768, ragged=True),
        # one token of a large batch over every key of its long cache: bandwidth
        _win("win_decode_dense_b32_128k", "decode", 32, 1, 32, 2, 131072, 0, Lmax=131072, ragged=True),
        # training: a padded batch with a short window, and one long sequence
        _win("win_backward_4k", "backward", 3, 4000, 16, 2, 257, 4, ragged=True),
        _win("win_backward_32k", "backward", 1, 32768, 32, 2, 4096, 64),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """Another case of the listed ones' ranges."""
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([g for g in (1, 2, 4, 8, 16) if Hkv * g <= 32])
    op, kind = rng.choice([("rope", "decode"), ("rope", "fresh"), ("rope", "chunk"), ("rope", "backward"),
                           ("win", "prefill"), ("win", "prefill"), ("win", "chunk"), ("win", "decode"),
                           ("win", "decode"), ("win", "backward"), ("win", "backward")])
    if op == "rope":
        rot, inter, wt = rng.choice([32, 64, 96, 128, 128]), rng.random() < 0.4, rng.choice(["bf16", "fp32"])
        if kind == "decode":
            return {**_rope("", kind, _logint(rng, 1, 64), 1, Hq, Hkv, rot, inter, _logint(rng, 64, 65536), False, wt)}
        B = rng.choice([1, 2, 3, 5])
        L = _logint(rng, 17, 65536 // B)
        Lmax = L + _logint(rng, 1, 16384) if kind == "chunk" else 0
        c = _rope("", kind, B, L, Hq, Hkv, rot, inter, Lmax, kind == "chunk", wt)
    else:
        n_sink = rng.choice([0, 1, 4, 64, 100])
        if kind == "decode":
            B = _logint(rng, 1, 48)
            Lmax = _logint(rng, 64, 131072)
            c = _win("", kind, B, 1, Hq, Hkv, _logint(rng, 16, 2 * Lmax), n_sink, Lmax, True)
        else:
            B = rng.choice([1, 1, 2, 3])
            if kind == "chunk":
                Lmax = _logint(rng, 300, 65536)
                L = _logint(rng, 1, min(Lmax, 4096))
                c = _win("", kind, B, L, Hq, Hkv, _logint(rng, 64, Lmax), n_sink, Lmax, True)
            else:
                L = _logint(rng, 100, 32768 // B)
                c = _win("", kind, B, L, Hq, Hkv, _logint(rng, 32, min(2 * L, 8192)), n_sink, 0,
                         kind == "backward" and rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, mul=1.0, add=0.0):
    # drawn in slices: a 128K cache batch has no fp32 copy of its own
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        n = min(1 << 27, flat.numel() - i)
        flat[i:i + n] = (torch.randn(n, generator=g, device="cuda") * mul + add).to(torch.bfloat16)
    return out


def _ints(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _table(n, rot):
    # cos in the first half of a row, sin in the second: angles in fp64, rounded once
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([torch.cos(ang), torch.sin(ang)], dim=1).to(torch.float32)


def prepare(case, seed):
    g = _gen(seed)
    B, L, Hq, Hkv = case["B"], case["L"], case["Hq"], case["Hkv"]
    s = {"case": case}
    if own:
        from trainable_block_sparse_compress_b200 import ops
        s["ops"] = ops
        s["p"] = ops.Params(batch=B, num_q_heads=Hq, num_kv_heads=Hkv)
    if case["op"] == "rope":
        kind, Lmax = case["kind"], case["Lmax"]
        wt = torch.bfloat16 if case["wtype"] == "bf16" else torch.float32
        # projection outputs: q, k and v are views of one packed row per token
        qkv = _randn(g, B, L, Hq + 2 * Hkv, D, mul=1.7)
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        s["qw"] = _randn(g, D, mul=0.2, add=1.0).to(wt)
        s["kw"] = _randn(g, D, mul=0.2, add=1.0).to(wt)
        s["eps"] = 1e-6
        s["starts"] = s["q_lens"] = None
        s["table"] = _table(max(L, Lmax), case["rot"])
        if kind == "decode":
            s["starts"] = _ints(g, B, 0, Lmax - 1)
            s["lens_out"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        if kind == "chunk":
            s["starts"] = _ints(g, B, 0, Lmax - L)
            s["q_lens"] = _ints(g, B, 0, L)
            s["q_out"] = torch.zeros(B, L, Hq, D, dtype=torch.bfloat16, device="cuda")
            s["k_cache"] = torch.zeros(B, Hkv, Lmax, D, dtype=torch.bfloat16, device="cuda")
            s["v_cache"] = torch.zeros(B, Hkv, Lmax, D, dtype=torch.bfloat16, device="cuda")
        if kind == "backward":
            s["dq"] = _randn(g, B, L, Hq, D)
            s["dk"] = _randn(g, B, Hkv, L, D)
            s["dv"] = _randn(g, B, Hkv, L, D)
        if own:
            s["starts_h"] = s["q_lens_h"] = None
        else:
            s["starts_h"] = s["starts"].tolist() if s["starts"] is not None else [0] * B
            s["q_lens_h"] = s["q_lens"].tolist() if s["q_lens"] is not None else [L] * B
        return s
    kind = case["kind"]
    Lmax = case["Lmax"] or L
    s["q"] = _randn(g, B, L, Hq, D)
    k = _randn(g, B, Hkv, Lmax, D)
    # neighbouring keys share an offset, as the keys of one passage do
    off = 0.5 * torch.randn(B, Hkv, (Lmax + 63) // 64, D, generator=g, device="cuda")
    for b in range(B):
        k[b] += off[b].repeat_interleave(64, dim=1)[:, :Lmax].to(torch.bfloat16)
    s["k"], s["v"] = k, _randn(g, B, Hkv, Lmax, D)
    s["q_lens"] = s["kv_lens"] = None
    ql, kl = [L] * B, [Lmax] * B
    if kind == "chunk":
        s["kv_lens"] = _ints(g, B, max(Lmax // 2, L), Lmax)
        s["q_lens"] = _ints(g, B, 1, L)
        ql, kl = s["q_lens"].tolist(), s["kv_lens"].tolist()
    elif kind == "decode":
        s["kv_lens"] = _ints(g, B, max(Lmax // 2, 1), Lmax)
        kl = s["kv_lens"].tolist()
        s["q"] = s["q"].view(B, Hq, D)
    elif kind == "backward" and case["ragged"]:
        s["q_lens"] = _ints(g, B, L // 2, L)
        ql = kl = s["q_lens"].tolist()
    s["ql"], s["kl"] = ql, kl
    if kind == "chunk":  # padding rows stay as they are: the caller's buffers
        s["o"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(B, Hq, L, dtype=torch.float32, device="cuda")
    if kind == "backward":
        s["do"] = _randn(g, B, L, Hq, D)
        s["o"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(B, Hq, L, dtype=torch.float32, device="cuda")
        for b in range(B):
            n = ql[b]
            o, lse = _attend(s["q"][b, :n], s["k"][b, :, :n], s["v"][b, :, :n], 0, case["window"], case["n_sink"])
            s["o"][b, :n], s["lse"][b, :, :n] = o.to(torch.bfloat16), lse
        for n, t in (("gq", s["q"]), ("gk", k), ("gv", k)):
            s[n] = torch.zeros_like(t)
    return s


# ------------------------------------------------------------------------ plain forms
def _norm_rope(x, w, eps, cs, rot, interleaved):
    """x [..., T, H, D] fp32, cs [T, rot] -> normalised, scaled and rotated."""
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w
    return _rotate(y, cs, rot, interleaved, 1.0)


def _rotate(y, cs, rot, interleaved, sign):
    h = rot // 2
    c, s = cs[:, None, :h], cs[:, None, h:] * sign
    out = y.clone()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * c - b * s, a * s + b * c
    else:
        a, b = y[..., :h], y[..., h:rot]
        out[..., :h], out[..., h:rot] = a * c - b * s, a * s + b * c
    return out


def _plain_rope(s):
    case = s["case"]
    B, L, kind, rot, inter = case["B"], case["L"], case["kind"], case["rot"], case["interleaved"]
    qw, kw, eps = s["qw"].float(), s["kw"].float(), s["eps"]
    if kind == "backward":
        cs = s["table"][:L]
        dqkv = []
        dws = []
        for x, w, dy in ((s["q"], qw, s["dq"]), (s["k"], kw, s["dk"].transpose(1, 2))):
            x, g = x.float(), _rotate(dy.float(), cs, rot, inter, -1.0)
            r = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
            xh = x * r
            dws.append((g * xh).sum((0, 1, 2), dtype=torch.float64).float())
            gw = g * w
            dqkv.append((r * (gw - xh * (gw * xh).mean(-1, keepdim=True))).to(torch.bfloat16))
        return dqkv[0], dqkv[1], s["dv"].transpose(1, 2).contiguous(), dws[0], dws[1]
    if kind == "chunk":
        qo, ko, vo = s["q_out"], s["k_cache"], s["v_cache"]
    else:
        qo = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
        ko = torch.empty((B, case["Hkv"], L, D), dtype=torch.bfloat16, device="cuda")
        vo = torch.empty_like(ko)
    for b in range(B):
        n, t0 = s["q_lens_h"][b], s["starts_h"][b]
        cs = s["table"][t0:t0 + n]
        at = t0 if kind == "chunk" else 0
        qo[b, :n] = _norm_rope(s["q"][b, :n].float(), qw, eps, cs, rot, inter).to(torch.bfloat16)
        ko[b, :, at:at + n] = _norm_rope(s["k"][b, :n].float(), kw, eps, cs, rot,
                                         inter).to(torch.bfloat16).transpose(0, 1)
        vo[b, :, at:at + n] = s["v"][b, :n].transpose(0, 1)
    if kind == "decode":
        s["lens_out"].copy_(s["starts"] + 1)
        return qo, ko, vo, s["lens_out"]
    return qo, ko, vo


def _tiles(R, t0, window, n_sink, rows):
    """Blocks of query rows with the keys that any of them sees: (r0, r1, key index tensor)."""
    for r0 in range(0, R, rows):
        r1 = min(R, r0 + rows)
        lo, hi = max(0, t0 + r0 - window + 1), t0 + r1
        keys = torch.arange(lo, hi, device="cuda")
        if min(n_sink, lo) > 0:
            keys = torch.cat([torch.arange(0, min(n_sink, lo), device="cuda"), keys])
        yield r0, r1, keys


def _visible(r0, r1, t0, keys, window, n_sink):
    t = torch.arange(t0 + r0, t0 + r1, device="cuda")[:, None]
    return (keys[None, :] <= t) & ((keys[None, :] > t - window) | (keys[None, :] < n_sink))


def _rows(R, Hq, N):
    return max(16, min(1024, (1 << 28) // (Hq * max(N, 1))))


def _attend(q, k, v, t0, window, n_sink):
    """q [R, Hq, D] at positions t0.., k, v [Hkv, N, D] -> o fp32 [R, Hq, D], lse fp32 [Hq, R]."""
    R, Hq, _ = q.shape
    Hkv, N, _ = k.shape
    G = Hq // Hkv
    o = torch.empty((R, Hq, D), dtype=torch.float32, device="cuda")
    lse = torch.empty((Hq, R), dtype=torch.float32, device="cuda")
    for r0, r1, keys in _tiles(R, t0, window, n_sink, _rows(R, Hq, min(N, window + 1024))):
        T = r1 - r0
        qb = q[r0:r1].float().view(T, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * T, D)
        kb, vb = k[:, keys].float(), v[:, keys].float()
        x = (qb @ kb.transpose(1, 2) * (D ** -0.5)).view(Hkv, G, T, -1)
        x = x.masked_fill(~_visible(r0, r1, t0, keys, window, n_sink), float("-inf"))
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - m)
        z = e.sum(-1, keepdim=True)
        ob = (e / z).view(Hkv, G * T, -1) @ vb
        o[r0:r1] = ob.view(Hkv, G, T, D).permute(2, 0, 1, 3).reshape(T, Hq, D)
        lse[:, r0:r1] = (m + torch.log(z)).view(Hq, T)
    return o, lse


def _attend_backward(q, k, v, o, lse, do, window, n_sink):
    R, Hq, _ = q.shape
    Hkv, N, _ = k.shape
    G = Hq // Hkv
    dq = torch.empty((R, Hq, D), dtype=torch.float32, device="cuda")
    dk = torch.zeros((Hkv, N, D), dtype=torch.float32, device="cuda")
    dv = torch.zeros_like(dk)
    sc = D ** -0.5
    for r0, r1, keys in _tiles(R, 0, window, n_sink, _rows(R, Hq, min(N, window + 1024))):
        T = r1 - r0

        def rows(x):
            return x[r0:r1].float().view(T, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, G * T, D)
        qb, ob, gb = rows(q), rows(o), rows(do)
        kb, vb = k[:, keys].float(), v[:, keys].float()
        x = (qb @ kb.transpose(1, 2) * sc).view(Hkv, G, T, -1)
        x = torch.exp(x - lse[:, r0:r1].view(Hkv, G, T, 1))
        x = x.masked_fill(~_visible(r0, r1, 0, keys, window, n_sink), 0.0).view(Hkv, G * T, -1)
        dv.index_add_(1, keys, x.transpose(1, 2) @ gb)
        dp = gb @ vb.transpose(1, 2)
        ds = x * (dp - (gb * ob).sum(-1, keepdim=True)) * sc
        dk.index_add_(1, keys, ds.transpose(1, 2) @ qb)
        dq[r0:r1] = (ds @ kb).view(Hkv, G, T, D).permute(2, 0, 1, 3).reshape(T, Hq, D)
    return dq, dk, dv


def _plain_win(s):
    case = s["case"]
    B, kind, W, ns = case["B"], case["kind"], case["window"], case["n_sink"]
    bf = torch.bfloat16
    if kind == "backward":
        for b in range(B):
            n = s["ql"][b]
            dq, dk, dv = _attend_backward(s["q"][b, :n], s["k"][b, :, :n], s["v"][b, :, :n], s["o"][b, :n],
                                          s["lse"][b, :, :n], s["do"][b, :n], W, ns)
            s["gq"][b, :n], s["gk"][b, :, :n], s["gv"][b, :, :n] = dq.to(bf), dk.to(bf), dv.to(bf)
        return s["gq"], s["gk"], s["gv"]
    if kind == "chunk":
        o, lse = s["o"], s["lse"]
    else:
        o = torch.empty_like(s["q"])
        lse = torch.empty((B, case["Hq"]) + (() if kind == "decode" else (case["L"],)), device="cuda")
    for b in range(B):
        n, N = s["ql"][b], s["kl"][b]
        q = s["q"][b:b + 1] if kind == "decode" else s["q"][b, :n]
        ob, lb = _attend(q, s["k"][b, :, :N], s["v"][b, :, :N], N - n, W, ns)
        if kind == "decode":
            o[b], lse[b] = ob[0].to(bf), lb[:, 0]
        else:
            o[b, :n], lse[b, :, :n] = ob.to(bf), lb
    return o, lse


def run(s):
    if not own:
        return _plain_rope(s) if s["case"]["op"] == "rope" else _plain_win(s)
    ops, p, case = s["ops"], s["p"], s["case"]
    kind = case["kind"]
    if case["op"] == "rope":
        kw = dict(q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"], interleaved=case["interleaved"])
        if kind == "backward":
            return ops.qk_norm_rope_backward(p, s["q"], s["k"], s["dq"], s["dk"], s["dv"], s["table"], **kw)
        if kind == "chunk":
            return ops.qk_norm_rope(p, s["q"], s["k"], s["v"], s["table"], starts=s["starts"], q_lens=s["q_lens"],
                                    k_cache=s["k_cache"], v_cache=s["v_cache"], q_out=s["q_out"], **kw)
        if kind == "decode":
            out = ops.qk_norm_rope(p, s["q"], s["k"], s["v"], s["table"], starts=s["starts"],
                                   lens_out=s["lens_out"], **kw)
            return (*out, s["lens_out"])
        return ops.qk_norm_rope(p, s["q"], s["k"], s["v"], s["table"], **kw)
    w, ns = case["window"], case["n_sink"]
    if kind == "prefill":
        return ops.window_attn_prefill(p, s["q"], s["k"], s["v"], w, ns)
    if kind == "chunk":
        return ops.window_attn_chunk(p, s["q"], s["k"], s["v"], w, ns, q_lens=s["q_lens"], kv_lens=s["kv_lens"],
                                     out=s["o"], lse=s["lse"])
    if kind == "decode":
        return ops.window_attn_decode(p, s["q"], s["k"], s["v"], s["kv_lens"], w, ns)
    return ops.window_attn_backward(p, s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], w, ns, lens=s["q_lens"],
                                    dq=s["gq"], dk=s["gk"], dv=s["gv"])


# ------------------------------------------------------------------------------ work
def _pairs(first, n, window, n_sink):
    """Visible (query, key) pairs of one head: queries at positions first .. first + n - 1."""
    total = 0
    for t0 in range(first, first + n, 1 << 16):
        t = torch.arange(t0, min(t0 + (1 << 16), first + n), dtype=torch.int64)
        win = torch.clamp(t + 1, max=window)
        total += int((win + torch.clamp(t + 1 - win, max=n_sink)).sum())
    return total


def work(case):
    B, L, Hq, Hkv = case["B"], case["L"], case["Hq"], case["Hkv"]
    kind = case["kind"]
    if case["op"] == "rope":
        H = Hq + 2 * Hkv
        tok = B * L / 2 if kind == "chunk" else B * L  # chunk lengths are uniform over 0..L
        tab = min(tok, max(L, case["Lmax"])) * case["rot"] * 4
        if kind == "backward":
            return {"bytes": tok * (H * 2 + Hq + Hkv) * D * 2 + tab, "flops": tok * (Hq + Hkv) * D * 16}
        return {"bytes": tok * H * D * 2 * 2 + tab, "flops": tok * (Hq + Hkv) * D * 8}
    W, ns = case["window"], case["n_sink"]
    if kind in ("prefill", "backward"):
        n = L if not case["ragged"] else (3 * L) // 4  # padded lengths are uniform over L/2..L
        pairs = B * _pairs(0, n, W, ns)
        qb, kb = B * n * Hq * D * 2, B * n * Hkv * D * 2
        if kind == "prefill":
            return {"bytes": 2 * qb + 2 * kb + B * n * Hq * 4, "flops": 4 * D * Hq * pairs}
        return {"bytes": 4 * qb + 4 * kb + B * n * Hq * 4, "flops": 10 * D * Hq * pairs}
    Lmax = case["Lmax"]
    kv = (max(Lmax // 2, L) + Lmax) // 2  # cache lengths are uniform over Lmax/2..Lmax
    n = 1 if kind == "decode" else (L + 1) // 2
    keys = min(kv, W + n - 1)
    keys += min(ns, kv - keys)
    return {"bytes": B * (2 * n * Hq * D * 2 + n * Hq * 4 + keys * Hkv * D * 4),
            "flops": 4 * D * Hq * B * _pairs(kv - n, n, W, ns)}


# ----------------------------------------------------------------------------- exact
def exact(case, seed):
    """The definitions in fp64, head by head."""
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return _exact_rope(s) if case["op"] == "rope" else _exact_win(s)


def _pairs_of(rot, interleaved):
    i = torch.arange(rot // 2, device="cuda")
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def _exact_rope(s):
    case = s["case"]
    B, L, Hq, Hkv, kind, rot = case["B"], case["L"], case["Hq"], case["Hkv"], case["kind"], case["rot"]
    ia, ib = _pairs_of(rot, case["interleaved"])
    eps, h = s["eps"], rot // 2

    def turn(z, cs, back):
        # complex multiplication by cos + i sin (its conjugate on the way back)
        w = torch.complex(z[..., ia], z[..., ib]) * torch.complex(cs[:, :h], -cs[:, h:] if back else cs[:, h:])
        z = z.clone()
        z[..., ia], z[..., ib] = w.real, w.imag
        return z
    if kind == "backward":
        cs = s["table"][:L].double()
        out, dws = [], []
        for x, w, dy, H in ((s["q"], s["qw"], s["dq"].transpose(1, 2), Hq), (s["k"], s["kw"], s["dk"], Hkv)):
            w = w.double()
            dx = torch.empty((B, L, H, D), dtype=torch.float64, device="cuda")
            dw = torch.zeros(D, dtype=torch.float64, device="cuda")
            for b in range(B):
                for j in range(H):
                    xj, g = x[b, :, j].double(), turn(dy[b, j].double(), cs, True)
                    ms = xj.pow(2).sum(-1) / D + eps
                    dw += (g * xj / ms.sqrt()[:, None]).sum(0)
                    gw = g * w
                    dot = (gw * xj).sum(-1) / D
                    dx[b, :, j] = gw / ms.sqrt()[:, None] - xj * (dot / ms.pow(1.5))[:, None]
            out.append(dx)
            dws.append(dw)
        return out[0], out[1], s["dv"].transpose(1, 2).contiguous(), dws[0], dws[1]
    Lo = case["Lmax"] if kind == "chunk" else L
    qo = torch.zeros((B, L, Hq, D), dtype=torch.float64, device="cuda")
    ko = torch.zeros((B, Hkv, Lo, D), dtype=torch.float64, device="cuda")
    vo = torch.zeros((B, Hkv, Lo, D), dtype=torch.bfloat16, device="cuda")
    for b in range(B):
        n, t0 = s["q_lens_h"][b], s["starts_h"][b]
        at = t0 if kind == "chunk" else 0
        cs = s["table"][t0:t0 + n].double()
        for x, w, H in ((s["q"], s["qw"], Hq), (s["k"], s["kw"], Hkv)):
            for j in range(H):
                xj = x[b, :n, j].double()
                y = turn(xj / (xj.pow(2).sum(-1, keepdim=True) / D + eps).sqrt() * w.double(), cs, False)
                if H == Hq and x is s["q"]:
                    qo[b, :n, j] = y
                else:
                    ko[b, j, at:at + n] = y
        for j in range(Hkv):
            vo[b, j, at:at + n] = s["v"][b, :n, j]
    if kind == "decode":
        return qo, ko, vo, s["starts"] + 1
    return qo, ko, vo


def _exact_win(s):
    case = s["case"]
    B, L, Hq, Hkv, kind = case["B"], case["L"], case["Hq"], case["Hkv"], case["kind"]
    W, ns, G = case["window"], case["n_sink"], case["Hq"] // case["Hkv"]
    f64 = torch.float64
    Lmax = s["k"].shape[2]
    q = s["q"].view(B, L, Hq, D)
    bwd = kind == "backward"
    o = torch.zeros((B, L, Hq, D), dtype=f64, device="cuda")
    lse = torch.zeros((B, Hq, L), dtype=f64, device="cuda")
    if bwd:
        gk = torch.zeros((B, Hkv, Lmax, D), dtype=f64, device="cuda")
        gv = torch.zeros_like(gk)
    for b in range(B):
        n, N = s["ql"][b], s["kl"][b]
        first = N - n
        step = max(16, min(2048, (1 << 26) // (G * min(N, W + 2048))))
        for j in range(Hkv):
            heads = slice(j * G, (j + 1) * G)
            for r0 in range(0, n, step):
                r1 = min(n, r0 + step)
                t = torch.arange(first + r0, first + r1, device="cuda")
                a = max(0, first + r0 - W + 1)
                segs = [(0, min(ns, a))] if min(ns, a) > 0 else []
                segs.append((a, first + r1))
                u = torch.cat([torch.arange(x, y, device="cuda") for x, y in segs])
                kk = torch.cat([s["k"][b, j, x:y] for x, y in segs]).to(f64)
                vv = torch.cat([s["v"][b, j, x:y] for x, y in segs]).to(f64)
                age = t[:, None] - u[None, :]
                ok = (age >= 0) & ((age < W) | (u < ns)[None, :])
                x = torch.matmul(q[b, r0:r1, heads].transpose(0, 1).to(f64), kk.t()) / math.sqrt(D)
                x = torch.where(ok, x, torch.full((), -math.inf, dtype=f64, device="cuda"))
                if not bwd:
                    z = torch.logsumexp(x, -1)
                    lse[b, heads, r0:r1] = z
                    o[b, r0:r1, heads] = torch.matmul(torch.exp(x - z[..., None]), vv).transpose(0, 1)
                    continue
                pr = torch.exp(x - s["lse"][b, heads, r0:r1, None].to(f64))
                go = s["do"][b, r0:r1, heads].transpose(0, 1).to(f64)
                dd = (go * s["o"][b, r0:r1, heads].transpose(0, 1).to(f64)).sum(-1, keepdim=True)
                ds = pr * (torch.matmul(go, vv.t()) - dd) / math.sqrt(D)
                o[b, r0:r1, heads] = torch.matmul(ds, kk).transpose(0, 1)  # dq
                dkk = torch.einsum("gtu,gtd->ud", ds, q[b, r0:r1, heads].transpose(0, 1).to(f64))
                dvv = torch.einsum("gtu,gtd->ud", pr, go)
                i = 0
                for x0, y0 in segs:
                    gk[b, j, x0:y0] += dkk[i:i + y0 - x0]
                    gv[b, j, x0:y0] += dvv[i:i + y0 - x0]
                    i += y0 - x0
    if bwd:
        return o, gk, gv
    if kind == "decode":
        return o.view(B, Hq, D), lse.view(B, Hq)
    return o, lse
