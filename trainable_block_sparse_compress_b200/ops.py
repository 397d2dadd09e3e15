"""Python binding of the InfLLM v2 C ABI: the same calls, taking torch tensors.

PyTorch provides device memory and the current CUDA stream; the binding checks shapes,
dtypes and devices, allocates outputs and workspaces with the caching allocator, and
passes raw pointers to the library.  No arithmetic of the method runs here.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional, Tuple

import torch

from . import _lib


def _is_i32(n) -> bool:
    """Whether the library's 32-bit argument can hold n (ctypes would cut a larger one)."""
    return -0x80000000 <= n <= 0x7fffffff


@dataclass(frozen=True)
class Params:
    batch: int
    num_q_heads: int
    num_kv_heads: int
    head_dim: int = 128
    block_size: int = 64
    kernel_size: int = 32
    kernel_stride: int = 16
    topk: int = 96
    n_init: int = 1
    n_local: int = 2
    softmax_scale: float = 0.0
    score_mode: int = 0  # 0 softmax-sum, 1 logit-sum (the block score)
    pool_mode: int = 0   # 0 overlapping kernels, 1 kernels inside the block (the pooling)

    @property
    def group(self) -> int:
        return self.num_q_heads // self.num_kv_heads

    def c(self) -> _lib.CParams:
        """The C struct, made once (the fields are frozen; the library only reads it)."""
        c = self.__dict__.get("_c")
        if c is None:
            for name, kind in _lib.CParams._fields_:
                if kind is ctypes.c_int32 and not _is_i32(getattr(self, name)):
                    raise _lib.InfLLMv2Error("infllmv2_check_params", _lib.ERR_INVALID_ARG)
            c = _lib.CParams(self.batch, self.num_q_heads, self.num_kv_heads, self.head_dim, self.block_size,
                             self.kernel_size, self.kernel_stride, self.topk, self.n_init, self.n_local,
                             float(self.softmax_scale), int(self.score_mode), int(self.pool_mode))
            self.__dict__["_c"] = c
        return c

    @staticmethod
    def from_workload(wl, batch: Optional[int] = None) -> "Params":
        return Params(batch if batch is not None else wl.batch, wl.num_q_heads, wl.num_kv_heads, wl.head_dim,
                      wl.block_size, wl.kernel_size, wl.kernel_stride, wl.topk, wl.n_init, wl.n_local)


def num_kernels(p: Params, n: int) -> int:
    return int(_lib.load().infllmv2_num_kernels(ctypes.byref(p.c()), n))


def num_blocks(p: Params, n: int) -> int:
    return (n + p.block_size - 1) // p.block_size


def workspace_size(p: Params, op: int, L: int) -> int:
    if not _is_i32(L):
        raise _lib.InfLLMv2Error("infllmv2_workspace_size", _lib.ERR_INVALID_ARG)
    v = int(_lib.load().infllmv2_workspace_size(ctypes.byref(p.c()), op, L))
    if v == ctypes.c_size_t(-1).value:
        raise _lib.InfLLMv2Error("infllmv2_workspace_size", _lib.ERR_INVALID_ARG)
    return v


def _workspace_bytes(p: Params, op: int, L: int) -> int:
    """workspace_size, remembered per problem (a function of the sizes and the device alone)."""
    sizes = p.__dict__.get("_ws")
    if sizes is None:
        sizes = p.__dict__["_ws"] = {}
    key = (op, L, _current_device())
    n = sizes.get(key)
    if n is None:
        if len(sizes) >= 256:
            sizes.clear()
        n = sizes[key] = workspace_size(p, op, L)
    return n


# The binding's own time bounds the smallest calls (a decode token's GPU work is a few us), so
# the current device and stream are read without building torch objects where torch offers it.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream() -> int:
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_current_device())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype, shape=None):
    # (a host tensor's get_device() is -1: it ends the comparison before a device is asked for)
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and 0 <= t.get_device() == _current_device():
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != _current_device():
        # the library launches on the current device: another device's pointer is not its memory
        raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _workspace(p: Params, op: int, L: int, ws: Optional[torch.Tensor], like: torch.Tensor) -> Optional[torch.Tensor]:
    """`ws` (any dtype and shape), or a fresh workspace where it is None or too small."""
    if ws is not None:
        _need(ws, "ws", ws.dtype, ws.shape)
    n = _workspace_bytes(p, op, L)
    if n == 0:
        return ws
    if ws is None or ws.numel() * ws.element_size() < n:
        ws = like.new_empty(n, dtype=torch.uint8)
    return ws


def compress_keys(p: Params, k: torch.Tensor, lens: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Semantic kernels: k bf16 [B, Hkv, Lmax, d] -> kc bf16 [B, Hkv, NK(Lmax), d]."""
    B, H, Lmax, d = k.shape
    _need(k, "k", torch.bfloat16, (p.batch, p.num_kv_heads, Lmax, p.head_dim))
    if lens is not None:
        _need(lens, "lens", torch.int32, (p.batch,))
    nk = num_kernels(p, Lmax)
    if out is None:
        out = torch.empty((B, H, nk, d), dtype=torch.bfloat16, device=k.device)
    _need(out, "kc", torch.bfloat16, (B, H, nk, d))
    st = _lib.load().infllmv2_compress_keys(ctypes.byref(p.c()), _ptr(k), _ptr(lens), Lmax, _ptr(out), _stream())
    _lib.check("infllmv2_compress_keys", st)
    return out


def select_blocks_prefill(p: Params, q: torch.Tensor, kc: torch.Tensor,
                          out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """q bf16 [B, L, Hq, d], kc [B, Hkv, NK(L), d] -> block_idx int32 [B, Hkv, L, topk]."""
    B, L, Hq, d = q.shape
    _need(q, "q", torch.bfloat16, (p.batch, L, p.num_q_heads, p.head_dim))
    _need(kc, "kc", torch.bfloat16, (p.batch, p.num_kv_heads, num_kernels(p, L), p.head_dim))
    if out is None:
        out = torch.empty((B, p.num_kv_heads, L, p.topk), dtype=torch.int32, device=q.device)
    _need(out, "block_idx", torch.int32, (B, p.num_kv_heads, L, p.topk))
    st = _lib.load().infllmv2_select_blocks(ctypes.byref(p.c()), _lib.MODE_PREFILL, _ptr(q), _ptr(kc), None, L,
                                            _ptr(out), None, 0, _stream())
    _lib.check("infllmv2_select_blocks", st)
    return out


def select_blocks_chunk(p: Params, q: torch.Tensor, kc: torch.Tensor, Lmax: int,
                        q_lens: Optional[torch.Tensor] = None, kv_lens: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Selection for a chunk of queries against existing caches.  q bf16 [B, Lq, Hq, d]: rows
    0..q_lens[b]-1 are the last q_lens[b] of kv_lens[b] cached tokens of sequence b (None:
    Lq and Lmax); kc [B, Hkv, NK(Lmax), d] -> block_idx int32 [B, Hkv, Lq, topk] (padding
    rows are not written)."""
    B, Lq, Hq, d = q.shape
    _need(q, "q", torch.bfloat16, (p.batch, Lq, p.num_q_heads, p.head_dim))
    _need(kc, "kc", torch.bfloat16, (p.batch, p.num_kv_heads, num_kernels(p, Lmax), p.head_dim))
    for t, name in ((q_lens, "q_lens"), (kv_lens, "kv_lens")):
        if t is not None:
            _need(t, name, torch.int32, (p.batch,))
    if out is None:
        out = torch.empty((B, p.num_kv_heads, Lq, p.topk), dtype=torch.int32, device=q.device)
    _need(out, "block_idx", torch.int32, (B, p.num_kv_heads, Lq, p.topk))
    st = _lib.load().infllmv2_select_blocks_chunk(ctypes.byref(p.c()), _ptr(q), Lq, _ptr(kc), _ptr(q_lens),
                                                  _ptr(kv_lens), Lmax, _ptr(out), None, 0, _stream())
    _lib.check("infllmv2_select_blocks_chunk", st)
    return out


def select_blocks_decode(p: Params, q: torch.Tensor, kc: torch.Tensor, lens: torch.Tensor, Lmax: int,
                         out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """q bf16 [B, Hq, d], kc [B, Hkv, NK(Lmax), d], lens int32 [B] -> int32 [B, Hkv, 1, topk]."""
    _need(q, "q", torch.bfloat16, (p.batch, p.num_q_heads, p.head_dim))
    _need(kc, "kc", torch.bfloat16, (p.batch, p.num_kv_heads, num_kernels(p, Lmax), p.head_dim))
    _need(lens, "lens", torch.int32, (p.batch,))
    if out is None:
        out = torch.empty((p.batch, p.num_kv_heads, 1, p.topk), dtype=torch.int32, device=q.device)
    _need(out, "block_idx", torch.int32, (p.batch, p.num_kv_heads, 1, p.topk))
    ws = _workspace(p, _lib.OP_SELECT_DECODE, Lmax, ws, q)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = _lib.load().infllmv2_select_blocks(ctypes.byref(p.c()), _lib.MODE_DECODE, _ptr(q), _ptr(kc), _ptr(lens),
                                            Lmax, _ptr(out), _ptr(ws), nbytes, _stream())
    _lib.check("infllmv2_select_blocks", st)
    return out


def sparse_attn_prefill(p: Params, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_idx: torch.Tensor,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        want_lse: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """O bf16 [B, L, Hq, d] and lse fp32 [B, Hq, L] over the selected blocks."""
    B, L, Hq, d = q.shape
    _need(q, "q", torch.bfloat16, (p.batch, L, p.num_q_heads, p.head_dim))
    _need(k, "k", torch.bfloat16, (p.batch, p.num_kv_heads, L, p.head_dim))
    _need(v, "v", torch.bfloat16, (p.batch, p.num_kv_heads, L, p.head_dim))
    _need(block_idx, "block_idx", torch.int32, (p.batch, p.num_kv_heads, L, p.topk))
    if out is None:
        out = torch.empty_like(q)
    _need(out, "o", torch.bfloat16, tuple(q.shape))
    if want_lse and lse is None:
        lse = torch.empty((B, Hq, L), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, Hq, L))
    st = _lib.load().infllmv2_sparse_attn_prefill(ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(block_idx),
                                                  L, _ptr(out), _ptr(lse), None, 0, _stream())
    _lib.check("infllmv2_sparse_attn_prefill", st)
    return out, lse


def sparse_attn_chunk(p: Params, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, block_idx: torch.Tensor,
                      q_lens: Optional[torch.Tensor] = None, kv_lens: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      want_lse: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention of a chunk of queries (as select_blocks_chunk) over caches k, v bf16
    [B, Hkv, Lmax, d]: O bf16 [B, Lq, Hq, d], lse fp32 [B, Hq, Lq] (padding rows not written)."""
    B, Lq, Hq, d = q.shape
    Lmax = k.shape[2]
    _need(q, "q", torch.bfloat16, (p.batch, Lq, p.num_q_heads, p.head_dim))
    _need(k, "k", torch.bfloat16, (p.batch, p.num_kv_heads, Lmax, p.head_dim))
    _need(v, "v", torch.bfloat16, (p.batch, p.num_kv_heads, Lmax, p.head_dim))
    _need(block_idx, "block_idx", torch.int32, (p.batch, p.num_kv_heads, Lq, p.topk))
    for t, name in ((q_lens, "q_lens"), (kv_lens, "kv_lens")):
        if t is not None:
            _need(t, name, torch.int32, (p.batch,))
    if out is None:
        out = torch.empty_like(q)
    _need(out, "o", torch.bfloat16, tuple(q.shape))
    if want_lse and lse is None:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, Hq, Lq))
    st = _lib.load().infllmv2_sparse_attn_chunk(ctypes.byref(p.c()), _ptr(q), Lq, _ptr(k), _ptr(v), _ptr(q_lens),
                                                _ptr(kv_lens), Lmax, _ptr(block_idx), _ptr(out), _ptr(lse), None, 0,
                                                _stream())
    _lib.check("infllmv2_sparse_attn_chunk", st)
    return out, lse


def sparse_attn_backward(p: Params, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                         lse: torch.Tensor, d_o: torch.Tensor, block_idx: torch.Tensor,
                         ws: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of the prefill sparse attention with the block lists fixed: q, o, d_o bf16
    [B, L, Hq, d], k, v bf16 [B, Hkv, L, d], lse fp32 [B, Hq, L] from the forward ->
    dq [B, L, Hq, d], dk, dv [B, Hkv, L, d] (bf16)."""
    B, L, Hq, d = q.shape
    for t, name in ((q, "q"), (o, "o"), (d_o, "d_o")):
        _need(t, name, torch.bfloat16, (p.batch, L, p.num_q_heads, p.head_dim))
    for t, name in ((k, "k"), (v, "v")):
        _need(t, name, torch.bfloat16, (p.batch, p.num_kv_heads, L, p.head_dim))
    _need(lse, "lse", torch.float32, (p.batch, p.num_q_heads, L))
    _need(block_idx, "block_idx", torch.int32, (p.batch, p.num_kv_heads, L, p.topk))
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    ws = _workspace(p, _lib.OP_ATTN_BACKWARD, L, ws, q)
    nbytes = ws.numel() * ws.element_size()
    st = _lib.load().infllmv2_sparse_attn_backward(ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                                   _ptr(d_o), _ptr(block_idx), L, _ptr(dq), _ptr(dk), _ptr(dv),
                                                   _ptr(ws), nbytes, _stream())
    _lib.check("infllmv2_sparse_attn_backward", st)
    return dq, dk, dv


def sparse_attn_decode(p: Params, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       lens: torch.Tensor, block_idx: torch.Tensor, out: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                       want_lse: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """O bf16 [B, Hq, d] and lse fp32 [B, Hq] for one query per sequence at lens[b]-1."""
    Lmax = k_cache.shape[2]
    _need(q, "q", torch.bfloat16, (p.batch, p.num_q_heads, p.head_dim))
    _need(k_cache, "k_cache", torch.bfloat16, (p.batch, p.num_kv_heads, Lmax, p.head_dim))
    _need(v_cache, "v_cache", torch.bfloat16, (p.batch, p.num_kv_heads, Lmax, p.head_dim))
    _need(lens, "lens", torch.int32, (p.batch,))
    _need(block_idx, "block_idx", torch.int32, (p.batch, p.num_kv_heads, 1, p.topk))
    if out is None:
        out = torch.empty_like(q)
    _need(out, "o", torch.bfloat16, tuple(q.shape))
    if want_lse and lse is None:
        lse = torch.empty((p.batch, p.num_q_heads), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, (p.batch, p.num_q_heads))
    ws = _workspace(p, _lib.OP_ATTN_DECODE, Lmax, ws, q)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = _lib.load().infllmv2_sparse_attn_decode(ctypes.byref(p.c()), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                                 _ptr(lens), Lmax, _ptr(block_idx), _ptr(out), _ptr(lse),
                                                 _ptr(ws), nbytes, _stream())
    _lib.check("infllmv2_sparse_attn_decode", st)
    return out, lse


def sparse_attn_decode_noalloc(p: Params, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                               lens: torch.Tensor, block_idx: torch.Tensor, out: torch.Tensor,
                               lse: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Decode attention for callers that cannot allocate device memory at call time: the
    caller passes preallocated outputs and the library uses its own fixed scratch array
    (no workspace).  Calls that overlap on the GPU race on that array."""
    Lmax = k_cache.shape[2]
    _need(q, "q", torch.bfloat16, (p.batch, p.num_q_heads, p.head_dim))
    _need(k_cache, "k_cache", torch.bfloat16, (p.batch, p.num_kv_heads, Lmax, p.head_dim))
    _need(v_cache, "v_cache", torch.bfloat16, (p.batch, p.num_kv_heads, Lmax, p.head_dim))
    _need(lens, "lens", torch.int32, (p.batch,))
    _need(block_idx, "block_idx", torch.int32, (p.batch, p.num_kv_heads, 1, p.topk))
    _need(out, "o", torch.bfloat16, tuple(q.shape))
    if lse is not None:
        _need(lse, "lse", torch.float32, (p.batch, p.num_q_heads))
    st = _lib.load().infllmv2_sparse_attn_decode_noalloc(ctypes.byref(p.c()), _ptr(q), _ptr(k_cache),
                                                         _ptr(v_cache), _ptr(lens), Lmax, _ptr(block_idx),
                                                         _ptr(out), _ptr(lse), _stream())
    _lib.check("infllmv2_sparse_attn_decode_noalloc", st)
    return out, lse


def append_kv(p: Params, k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              lens: torch.Tensor, kc: torch.Tensor) -> None:
    """Appends one token per sequence: k_new / v_new bf16 [B, Hkv, d] go to position lens[b]
    of the caches [B, Hkv, Lmax, d], a completed semantic kernel goes to kc
    [B, Hkv, NK(Lmax), d], and lens (int32 [B], on the GPU) is incremented in place."""
    Lmax = k_cache.shape[2]
    _need(k_new, "k_new", torch.bfloat16, (p.batch, p.num_kv_heads, p.head_dim))
    _need(v_new, "v_new", torch.bfloat16, (p.batch, p.num_kv_heads, p.head_dim))
    _need(k_cache, "k_cache", torch.bfloat16, (p.batch, p.num_kv_heads, Lmax, p.head_dim))
    _need(v_cache, "v_cache", torch.bfloat16, (p.batch, p.num_kv_heads, Lmax, p.head_dim))
    _need(lens, "lens", torch.int32, (p.batch,))
    _need(kc, "kc", torch.bfloat16, (p.batch, p.num_kv_heads, num_kernels(p, Lmax), p.head_dim))
    st = _lib.load().infllmv2_append_kv(ctypes.byref(p.c()), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(lens), Lmax, _ptr(kc), _stream())
    _lib.check("infllmv2_append_kv", st)


def rope_table(p: Params, inv_freq: torch.Tensor, n: int, scale: float = 1.0,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rotation table for positions 0..n-1: inv_freq fp32 [rot / 2] -> fp32 [n, rot], row t =
    scale cos(t f_i), then scale sin(t f_i), with the angles in fp64."""
    _need(inv_freq, "inv_freq", torch.float32)
    rot = 2 * inv_freq.numel()
    if out is None:
        out = torch.empty((n, rot), dtype=torch.float32, device=inv_freq.device)
    _need(out, "table", torch.float32, (n, rot))
    st = _lib.load().infllmv2_rope_table(ctypes.byref(p.c()), _ptr(inv_freq), rot, n, scale, _ptr(out), _stream())
    _lib.check("infllmv2_rope_table", st)
    return out


def _need_tokens(t: torch.Tensor, name: str, B: int, L: int, H: int, d: int) -> int:
    """Token rows [B, L, H, d] with contiguous [H, d] and one stride between consecutive tokens
    (a slice of a packed projection output is such a view).  Returns that stride."""
    if t.shape != (B, L, H, d):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(B, L, H, d)}")
    sb, sl, sh, sd = t.stride()
    # a stride over an axis of length 1 says nothing
    if not (t.dtype is torch.bfloat16 and sd == 1 and (sh == d or H == 1)
            and 0 <= t.get_device() == _current_device()):
        _need(t[:1, :1], name, torch.bfloat16)  # the heads of a token, as any other tensor
    if L > 1:
        stride = sl
    else:
        stride = sb if B > 1 else H * d
    if B > 1 and sb != L * stride:
        raise ValueError(f"{name} must have one stride between consecutive tokens, got {t.stride()}")
    return stride


def _norm_weights(p: Params, q_weight, k_weight) -> int:
    """Checks the norm weights ([d], both fp32 or both bf16, each may be None); 1 when fp32."""
    first = q_weight if q_weight is not None else k_weight
    if first is None:
        return 0
    dt = first.dtype
    if k_weight is not None and k_weight.dtype is not dt:
        raise ValueError("q_weight and k_weight must have one dtype")
    if dt not in (torch.float32, torch.bfloat16):
        raise ValueError(f"q_weight and k_weight must be torch.float32 or torch.bfloat16, got {dt}")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _need(w, name, dt, (p.head_dim,))
    return 1 if dt == torch.float32 else 0


def qk_norm_rope(p: Params, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, interleaved: bool = False, starts: Optional[torch.Tensor] = None,
                 q_lens: Optional[torch.Tensor] = None, k_cache: Optional[torch.Tensor] = None,
                 v_cache: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                 k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                 lens_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Per-head RMS norm of q and k and their position rotation, from the projection's rows to
    the attention's layouts.  q bf16 [B, Lq, Hq, d], k, v [B, Lq, Hkv, d] (views of one packed
    tensor allowed: only the token stride is free); table fp32 [n, rot] (rope_table); weights
    [d], fp32 or bf16, or None.  Row r of sequence b sits at position starts[b] + r (None: r);
    rows at or past q_lens[b] are padding.  Returns q [B, Lq, Hq, d] and k, v: with k_cache and
    v_cache [B, Hkv, Lmax, d], the caches with the rows written at their positions; otherwise
    [B, Hkv, Lq, d] (with Lq = 1, q[:, 0], k[:, :, 0] and v[:, :, 0] are what decode_step
    takes).  Rows of padding are zero in outputs made here and not written in those given.
    lens_out int32 [B], when given, receives starts[b] + the sequence's rows."""
    B, Lq = q.shape[:2]
    qs = _need_tokens(q, "q", p.batch, Lq, p.num_q_heads, p.head_dim)
    ks = _need_tokens(k, "k", p.batch, Lq, p.num_kv_heads, p.head_dim)
    vs = _need_tokens(v, "v", p.batch, Lq, p.num_kv_heads, p.head_dim)
    n, rot = table.shape
    _need(table, "table", torch.float32, (n, rot))
    wf = _norm_weights(p, q_weight, k_weight)
    if starts is not None:
        _need(starts, "starts", torch.int32, (B,))
    if q_lens is not None:
        _need(q_lens, "q_lens", torch.int32, (B,))
    if lens_out is not None:
        _need(lens_out, "lens_out", torch.int32, (B,))
    if (k_cache is None) != (v_cache is None):
        raise ValueError("k_cache and v_cache go together")
    # outputs made here need no checks; their rows of padding reach calls that take no lengths
    make = q.new_empty if q_lens is None else q.new_zeros
    if q_out is None:
        q_out = make((B, Lq, p.num_q_heads, p.head_dim))
    else:
        _need(q_out, "q_out", torch.bfloat16, (B, Lq, p.num_q_heads, p.head_dim))
    if k_cache is not None:
        if k_out is not None or v_out is not None:
            raise ValueError("k_out and v_out are for fresh outputs, without caches")
        Lout = k_cache.shape[2]
        for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
            _need(t, name, torch.bfloat16, (B, p.num_kv_heads, Lout, p.head_dim))
        k_out, v_out = k_cache, v_cache
    else:
        Lout = Lq
        kv_shape = (B, p.num_kv_heads, Lq, p.head_dim)
        if k_out is not None:
            _need(k_out, "k_out", torch.bfloat16, kv_shape)
        else:
            k_out = make(kv_shape)
        if v_out is not None:
            _need(v_out, "v_out", torch.bfloat16, kv_shape)
        else:
            v_out = make(kv_shape)
    st = _lib.load().infllmv2_qk_norm_rope(ctypes.byref(p.c()), _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, Lq,
                                           _ptr(q_weight), _ptr(k_weight), wf, eps, _ptr(table), n, rot,
                                           int(interleaved), _ptr(starts), _ptr(q_lens), _ptr(q_out), _ptr(k_out),
                                           _ptr(v_out), Lout, int(k_cache is not None), _ptr(lens_out), _stream())
    _lib.check("infllmv2_qk_norm_rope", st)
    return q_out, k_out, v_out


def qk_norm_rope_backward(p: Params, q: torch.Tensor, k: torch.Tensor, d_q: torch.Tensor, d_k: torch.Tensor,
                          d_v: torch.Tensor, table: torch.Tensor, q_weight: Optional[torch.Tensor] = None,
                          k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6, interleaved: bool = False,
                          starts: Optional[torch.Tensor] = None, q_lens: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """Gradients of qk_norm_rope's inputs: q, k as given to it, d_q bf16 [B, Lq, Hq, d], d_k, d_v
    [B, Hkv, Lq, d] (the layouts sparse_attn_backward and window_attn_backward return).  Returns
    (dq, dk, dv, d_qw, d_kw): token rows [B, Lq, H, d], views of one packed tensor
    [B, Lq, Hq + 2 Hkv, d] (`out`: rows of padding are not written; allocated when None: they are
    zero), and the weights' gradients, fp32 [d] (None for a weight that is None)."""
    B, Lq = q.shape[:2]
    Hq, Hkv, d = p.num_q_heads, p.num_kv_heads, p.head_dim
    qs = _need_tokens(q, "q", p.batch, Lq, Hq, d)
    ks = _need_tokens(k, "k", p.batch, Lq, Hkv, d)
    _need(d_q, "d_q", torch.bfloat16, (B, Lq, Hq, d))
    kv_shape = (B, Hkv, Lq, d)
    _need(d_k, "d_k", torch.bfloat16, kv_shape)
    _need(d_v, "d_v", torch.bfloat16, kv_shape)
    n, rot = table.shape
    _need(table, "table", torch.float32, (n, rot))
    wf = _norm_weights(p, q_weight, k_weight)
    if starts is not None:
        _need(starts, "starts", torch.int32, (B,))
    if q_lens is not None:
        _need(q_lens, "q_lens", torch.int32, (B,))
    if out is None:
        # the rows go into the projection's weight gradient: none may hold what was in memory
        make = q.new_empty if q_lens is None else q.new_zeros
        out = make((B, Lq, Hq + 2 * Hkv, d))
    else:
        _need(out, "out", torch.bfloat16, (B, Lq, Hq + 2 * Hkv, d))
    dq, dk, dv = out.split((Hq, Hkv, Hkv), 2)
    d_qw = None if q_weight is None else q.new_empty(d, dtype=torch.float32)
    d_kw = None if k_weight is None else q.new_empty(d, dtype=torch.float32)
    ws = _workspace(p, _lib.OP_QK_NORM_ROPE_BACKWARD, Lq, ws, q)
    nbytes = ws.numel() * ws.element_size()
    rs = (Hq + 2 * Hkv) * d
    st = _lib.load().infllmv2_qk_norm_rope_backward(
        ctypes.byref(p.c()), _ptr(q), qs, _ptr(k), ks, _ptr(d_q), _ptr(d_k), _ptr(d_v), Lq, _ptr(q_weight),
        _ptr(k_weight), wf, eps, _ptr(table), n, rot, int(interleaved), _ptr(starts), _ptr(q_lens), _ptr(dq), rs,
        _ptr(dk), rs, _ptr(dv), rs, _ptr(d_qw), _ptr(d_kw), _ptr(ws), nbytes, _stream())
    _lib.check("infllmv2_qk_norm_rope_backward", st)
    return dq, dk, dv, d_qw, d_kw


def _need_window(fn: str, window: int, n_sink: int) -> None:
    """The library's own check, made before the numbers become 32-bit arguments."""
    if not (1 <= window <= 0x7fffffff and 0 <= n_sink <= 0x7fffffff):
        raise _lib.InfLLMv2Error(fn, _lib.ERR_INVALID_ARG)


def window_attn_chunk(p: Params, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int, n_sink: int = 0,
                      q_lens: Optional[torch.Tensor] = None, kv_lens: Optional[torch.Tensor] = None,
                      out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      want_lse: bool = True,
                      ws: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Sliding-window attention of a chunk of queries (as sparse_attn_chunk: rows 0..q_lens[b]-1
    are the last q_lens[b] of kv_lens[b] cached tokens) over caches k, v bf16 [B, Hkv, Lmax, d]:
    the query at position t sees the keys u <= t with u > t - window or u < n_sink.  O bf16
    [B, Lq, Hq, d], lse fp32 [B, Hq, Lq] (padding rows not written; with q_lens those of an O made
    here are zero, as the output projection's weight gradient runs over them)."""
    _need_window("infllmv2_window_attn", window, n_sink)
    B, Lq, Hq, d = q.shape
    Lmax = k.shape[2]
    _need(q, "q", torch.bfloat16, (p.batch, Lq, p.num_q_heads, p.head_dim))
    kv_shape = (p.batch, p.num_kv_heads, Lmax, p.head_dim)
    _need(k, "k", torch.bfloat16, kv_shape)
    _need(v, "v", torch.bfloat16, kv_shape)
    if q_lens is not None:
        _need(q_lens, "q_lens", torch.int32, (p.batch,))
    if kv_lens is not None:
        _need(kv_lens, "kv_lens", torch.int32, (p.batch,))
    if out is None:
        out = torch.empty_like(q) if q_lens is None else torch.zeros_like(q)
    else:
        _need(out, "o", torch.bfloat16, q.shape)
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, Hq, Lq))
    elif want_lse:
        lse = q.new_empty((B, Hq, Lq), dtype=torch.float32)
    ws = _workspace(p, _lib.OP_WINDOW_ATTN, Lq, ws, q)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = _lib.load().infllmv2_window_attn(ctypes.byref(p.c()), _ptr(q), Lq, _ptr(k), _ptr(v), _ptr(q_lens),
                                          _ptr(kv_lens), Lmax, window, n_sink, _ptr(out), _ptr(lse), _ptr(ws), nbytes,
                                          _stream())
    _lib.check("infllmv2_window_attn", st)
    return out, lse


def window_attn_prefill(p: Params, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, window: int, n_sink: int = 0,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        want_lse: bool = True,
                        ws: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Sliding-window attention of fresh sequences: q bf16 [B, L, Hq, d], k, v [B, Hkv, L, d] ->
    O [B, L, Hq, d], lse fp32 [B, Hq, L].  window >= L is plain causal attention.  For a padded
    batch use window_attn_chunk with q_lens = kv_lens."""
    if k.shape[2] != q.shape[1]:
        raise ValueError(f"k holds {k.shape[2]} tokens, q {q.shape[1]}")
    return window_attn_chunk(p, q, k, v, window, n_sink, out=out, lse=lse, want_lse=want_lse, ws=ws)


def window_attn_decode(p: Params, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, lens: torch.Tensor,
                       window: int, n_sink: int = 0, out: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                       want_lse: bool = True) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Sliding-window attention of one token per sequence at position lens[b]-1: q bf16
    [B, Hq, d], caches [B, Hkv, Lmax, d] -> O [B, Hq, d], lse fp32 [B, Hq] (0 and -inf for an
    empty sequence)."""
    _need_window("infllmv2_window_attn_decode", window, n_sink)
    Lmax = k_cache.shape[2]
    _need(q, "q", torch.bfloat16, (p.batch, p.num_q_heads, p.head_dim))
    kv_shape = (p.batch, p.num_kv_heads, Lmax, p.head_dim)
    _need(k_cache, "k_cache", torch.bfloat16, kv_shape)
    _need(v_cache, "v_cache", torch.bfloat16, kv_shape)
    _need(lens, "lens", torch.int32, (p.batch,))
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "o", torch.bfloat16, q.shape)
    if lse is not None:
        _need(lse, "lse", torch.float32, (p.batch, p.num_q_heads))
    elif want_lse:
        lse = q.new_empty((p.batch, p.num_q_heads), dtype=torch.float32)
    ws = _workspace(p, _lib.OP_WINDOW_DECODE, Lmax, ws, q)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = _lib.load().infllmv2_window_attn_decode(ctypes.byref(p.c()), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                                 _ptr(lens), Lmax, window, n_sink, _ptr(out), _ptr(lse), _ptr(ws),
                                                 nbytes, _stream())
    _lib.check("infllmv2_window_attn_decode", st)
    return out, lse


def window_attn_backward(p: Params, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                         lse: torch.Tensor, d_o: torch.Tensor, window: int, n_sink: int = 0,
                         lens: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                         dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                         dv: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of the window attention over fresh sequences of lens[b] tokens (None: L): q, o,
    d_o bf16 [B, L, Hq, d], k, v bf16 [B, Hkv, L, d], lse fp32 [B, Hq, L] from the forward ->
    dq [B, L, Hq, d], dk, dv [B, Hkv, L, d] (bf16; rows of padding are not written in tensors that
    are given, and zero in those allocated here).  dq, dk and dv, when given, must not overlap
    q, k, v, d_o or one another."""
    _need_window("infllmv2_window_attn_backward", window, n_sink)
    B, L, Hq, d = q.shape
    for t, name in ((q, "q"), (o, "o"), (d_o, "d_o")):
        _need(t, name, torch.bfloat16, (p.batch, L, p.num_q_heads, p.head_dim))
    for t, name in ((k, "k"), (v, "v")):
        _need(t, name, torch.bfloat16, (p.batch, p.num_kv_heads, L, p.head_dim))
    _need(lse, "lse", torch.float32, (p.batch, p.num_q_heads, L))
    if lens is not None:
        _need(lens, "lens", torch.int32, (p.batch,))
    for t, ref, name in ((dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv")):
        if t is not None:
            _need(t, name, torch.bfloat16, ref.shape)
    make = torch.empty_like if lens is None else torch.zeros_like
    dq = make(q) if dq is None else dq
    dk = make(k) if dk is None else dk
    dv = make(v) if dv is None else dv
    ws = _workspace(p, _lib.OP_WINDOW_BACKWARD, L, ws, q)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = _lib.load().infllmv2_window_attn_backward(ctypes.byref(p.c()), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                                   _ptr(d_o), _ptr(lens), L, window, n_sink, _ptr(dq), _ptr(dk),
                                                   _ptr(dv), _ptr(ws), nbytes, _stream())
    _lib.check("infllmv2_window_attn_backward", st)
    return dq, dk, dv


def device_error(clear: bool = True) -> int:
    v = int(_lib.load().infllmv2_device_error(1 if clear else 0))
    if v < 0:
        raise _lib.InfLLMv2Error("infllmv2_device_error", v)
    return v


def prefill(p: Params, q, k, v):
    """Whole prefill path: compress -> select -> sparse attention.  Returns (o, lse, idx, kc)."""
    kc = compress_keys(p, k)
    idx = select_blocks_prefill(p, q, kc)
    o, lse = sparse_attn_prefill(p, q, k, v, idx)
    return o, lse, idx, kc


def prefill_chunk(p: Params, q, k_cache, v_cache, kc, q_lens=None, kv_lens=None):
    """A chunk of queries against filled caches (keys, values and semantic kernels of
    kv_lens[b] tokens each): select -> sparse attention.  Returns (o, lse, idx)."""
    Lmax = k_cache.shape[2]
    idx = select_blocks_chunk(p, q, kc, Lmax, q_lens=q_lens, kv_lens=kv_lens)
    o, lse = sparse_attn_chunk(p, q, k_cache, v_cache, idx, q_lens=q_lens, kv_lens=kv_lens)
    return o, lse, idx


def decode_step(p: Params, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, kc: torch.Tensor,
                lens: torch.Tensor, k_new: Optional[torch.Tensor] = None, v_new: Optional[torch.Tensor] = None,
                lens_out: Optional[torch.Tensor] = None, block_idx: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, want_lse: bool = True):
    """One decode step in one launch.  With k_new / v_new [B, Hkv, d]: the new token is
    appended at lens[b] (caches and kc updated in place) and lens_out[b] = lens[b] + 1
    (lens_out allocated when None); without: the query sits at lens[b]-1.  Then block
    selection and sparse attention over the selected blocks.  Returns (o, lse, block_idx)
    and, when appending, lens_out as a fourth element."""
    Lmax = k_cache.shape[2]
    _need(q, "q", torch.bfloat16, (p.batch, p.num_q_heads, p.head_dim))
    _need(k_cache, "k_cache", torch.bfloat16, (p.batch, p.num_kv_heads, Lmax, p.head_dim))
    _need(v_cache, "v_cache", torch.bfloat16, (p.batch, p.num_kv_heads, Lmax, p.head_dim))
    _need(kc, "kc", torch.bfloat16, (p.batch, p.num_kv_heads, num_kernels(p, Lmax), p.head_dim))
    _need(lens, "lens", torch.int32, (p.batch,))
    appending = k_new is not None or v_new is not None
    if appending:
        _need(k_new, "k_new", torch.bfloat16, (p.batch, p.num_kv_heads, p.head_dim))
        _need(v_new, "v_new", torch.bfloat16, (p.batch, p.num_kv_heads, p.head_dim))
        if lens_out is None:
            lens_out = torch.empty_like(lens)
        _need(lens_out, "lens_out", torch.int32, (p.batch,))
        if lens_out.data_ptr() == lens.data_ptr():
            raise ValueError("lens_out must not be lens")
    if block_idx is None:
        block_idx = torch.empty((p.batch, p.num_kv_heads, 1, p.topk), dtype=torch.int32, device=q.device)
    _need(block_idx, "block_idx", torch.int32, (p.batch, p.num_kv_heads, 1, p.topk))
    if out is None:
        out = torch.empty_like(q)
    _need(out, "o", torch.bfloat16, tuple(q.shape))
    if want_lse and lse is None:
        lse = torch.empty((p.batch, p.num_q_heads), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, (p.batch, p.num_q_heads))
    st = _lib.load().infllmv2_decode_step(ctypes.byref(p.c()), _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache),
                                          _ptr(v_cache), _ptr(kc), _ptr(lens), _ptr(lens_out), Lmax, _ptr(block_idx),
                                          _ptr(out), _ptr(lse), _stream())
    _lib.check("infllmv2_decode_step", st)
    if appending:
        return out, lse, block_idx, lens_out
    return out, lse, block_idx


def decode(p: Params, q, k_cache, v_cache, kc, lens, Lmax):
    """One decode step over a filled cache (Lmax = the caches' length): select -> sparse
    attention, fused in one launch.  Returns (o, lse, idx)."""
    assert k_cache.shape[2] == Lmax, "Lmax is the caches' length"
    return decode_step(p, q, k_cache, v_cache, kc, lens)
