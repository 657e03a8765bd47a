"""The caller's own decode and verification steps on a paged KV cache: append
keys and values (rotated on the way), attend behind shared prefixes, and
multiply by 4-bit weights.  Thin faces of dflash_append_kv,
dflash_prefix_attention and dflash_gemm_w4 (include/dflash.h states what each
computes, checks and refuses).

Work goes to `stream` (default: the current stream of the tensors' device);
temporary memory comes from PyTorch's allocator on that stream.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import _lib

_ELEM = {torch.float32: _lib.ELEM_F32, torch.bfloat16: _lib.ELEM_BF16, torch.float16: _lib.ELEM_F16}
_W4 = {"int4": _lib.W4_INT, "e2m1": _lib.W4_E2M1}


def _need(cond, what: str) -> None:
    if not cond:
        raise ValueError(what)


class _On:
    """The device of `dev`, and the stream the work goes to, as current ones."""

    def __init__(self, dev: torch.device, stream: Optional[torch.cuda.Stream]):
        _need(dev.type == "cuda", "tensors must be on a CUDA device")
        _need(stream is None or stream.device == dev, "the stream belongs to another device than the tensors")
        self.guard = None
        if stream is not None:
            self.guard = torch.cuda.stream(stream)
        elif torch.cuda.current_device() != dev.index:
            self.guard = torch.cuda.device(dev)

    def __enter__(self) -> int:
        if self.guard is not None:
            self.guard.__enter__()
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _ints(t: Optional[torch.Tensor], n: int, dev, what: str) -> Optional[int]:
    """The address of an optional int32 tensor of n entries."""
    if t is None:
        return None
    _need(t.dtype == torch.int32 and t.device == dev and t.numel() == n and t.is_contiguous(),
          f"{what}: contiguous int32 of {n} entries on the cache's device")
    return t.data_ptr()


def _status(t: Optional[torch.Tensor], dev) -> Optional[int]:
    return None if t is None else _ints(t, 1, dev, "status")


def _token_stride(t: torch.Tensor, what: str) -> int:
    """Elements between tokens of [B, T, heads, head_dim] with contiguous heads and evenly spaced tokens."""
    B, T, H, dh = t.shape
    sb, st, sh, sd = t.stride()
    _need(sd == 1 and (H == 1 or sh == dh), f"{what}: the heads of a token must be contiguous")
    if T == 1:
        return sb if B > 1 else H * dh
    _need(B == 1 or sb == T * st, f"{what}: tokens must be evenly spaced")
    return st


class PagedKV:
    """One layer of a paged KV cache in the caller's tensors: k, v
    [n_pages, n_kv_heads, 16, head_dim] (fp32, bf16 or fp16), page_table int32
    [n_seqs, max_pages], seq_len int32 [n_seqs]."""

    __slots__ = ("k", "v", "page_table", "seq_len", "view", "ref")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, seq_len: torch.Tensor):
        _need(k.dim() == 4 and k.shape == v.shape and k.shape[2] == 16, "k, v: [n_pages, n_kv_heads, 16, head_dim]")
        _need(k.dtype in _ELEM and v.dtype == k.dtype, "k, v: fp32, bf16 or fp16, both alike")
        _need(k.is_contiguous() and v.is_contiguous(), "k, v must be contiguous")
        _need(page_table.dim() == 2 and page_table.dtype == torch.int32 and page_table.is_contiguous(),
              "page_table: contiguous int32 [n_seqs, max_pages]")
        _need(seq_len.dtype == torch.int32 and seq_len.is_contiguous() and seq_len.numel() == page_table.shape[0],
              "seq_len: contiguous int32 [n_seqs]")
        dev = k.device
        _need(v.device == dev and page_table.device == dev and seq_len.device == dev, "one device for the whole cache")
        self.k, self.v, self.page_table, self.seq_len = k, v, page_table, seq_len
        n, h, _, dh = k.shape
        self.view = _lib.DflashPagedKV(k.data_ptr(), v.data_ptr(), page_table.data_ptr(), seq_len.data_ptr(), n,
                                       page_table.shape[0], page_table.shape[1], h, dh, _ELEM[k.dtype])
        self.ref = ctypes.byref(self.view)


def rope_table(rows: int, head_dim: int, theta: float, device="cuda", stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(cos, sin) fp32 [rows, head_dim / 2] of pos * theta^(-2i / head_dim)."""
    dev = torch.device(device)
    if dev.index is None:
        dev = torch.device(dev.type, torch.cuda.current_device())
    with _On(dev, stream) as s:
        cos, sin = (torch.empty((rows, head_dim // 2), dtype=torch.float32, device=dev) for _ in range(2))
        _lib.check(_lib.lib().dflash_rope_table(cos.data_ptr(), sin.data_ptr(), rows, head_dim, float(theta), s),
                   "dflash_rope_table")
    return cos, sin


def append_kv(kv: PagedKV, k: torch.Tensor, v: torch.Tensor, n_rows: Optional[torch.Tensor] = None, *,
              seq: Optional[torch.Tensor] = None, pos_base: Optional[torch.Tensor] = None,
              rope: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, q: Optional[torch.Tensor] = None,
              q_out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """The rows k, v [B, T, n_kv_heads, head_dim] as the last n_rows[b] tokens
    of sequence seq[b] (whose seq_len already counts them), keys rotated by
    `rope` = (cos, sin) at pos_base[b] + slot; q [B, T, n_q_heads, head_dim]
    rotated alike into q_out (cache type).  Returns q_out."""
    _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype and k.dtype in _ELEM,
          "k, v: [B, T, n_kv_heads, head_dim] of one type")
    B, T, H, dh = k.shape
    dev = kv.k.device
    _need(H == kv.k.shape[1] and dh == kv.k.shape[3], "k, v do not have the cache's heads")
    _need(k.device == dev and v.device == dev, "k, v are on another device than the cache")
    cos = sin = qp = op = None
    rows = ld_q = Hq = 0
    if rope is not None:
        c, s_ = rope
        rows = c.shape[0]
        _need(c.shape == s_.shape == (rows, dh // 2) and c.dtype == s_.dtype == torch.float32 and c.is_contiguous()
              and s_.is_contiguous() and c.device == dev and s_.device == dev,
              "rope: contiguous fp32 (cos, sin) [rows, head_dim / 2] on the cache's device")
        cos, sin = c.data_ptr(), s_.data_ptr()
    with _On(dev, stream) as s:
        if q is not None:
            _need(q.dim() == 4 and q.shape[:2] == (B, T) and q.shape[3] == dh and q.dtype == k.dtype
                  and q.device == dev, "q: [B, T, n_q_heads, head_dim], the type of k, on the cache's device")
            Hq = q.shape[2]
            if q_out is None:
                q_out = torch.empty((B, T, Hq, dh), dtype=kv.k.dtype, device=dev)
            _need(q_out.shape == q.shape and q_out.dtype == kv.k.dtype and q_out.is_contiguous()
                  and q_out.device == dev, "q_out: contiguous, the shape of q and the cache's type")
            qp, ld_q, op = q.data_ptr(), _token_stride(q, "q"), q_out.data_ptr()
        else:
            _need(q_out is None, "q_out without q")
        _lib.check(_lib.lib().dflash_append_kv(
            kv.ref, k.data_ptr(), _token_stride(k, "k"), v.data_ptr(), _token_stride(v, "v"), _ELEM[k.dtype],
            _ints(n_rows, B, dev, "n_rows"), _ints(seq, B, dev, "seq"), _ints(pos_base, B, dev, "pos_base"), B, T,
            cos, sin, rows, qp, ld_q, Hq, op, _status(status, dev), s), "dflash_append_kv")
    return q_out


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(n_pages, n_seqs, max_pages, Hkv, dh, elem, Hq, B, T, NG, max_prefix, max_len, dev):
    view = _lib.DflashPagedKV(256, 256, 256, 256, n_pages, n_seqs, max_pages, Hkv, dh, elem)
    return _lib.lib().dflash_prefix_attention_workspace(ctypes.byref(view), Hq, B, T, NG, max_prefix, max_len)


def prefix_attention_workspace(kv: PagedKV, n_q_heads: int, B: int, T: int, n_groups: int, max_prefix: int = 0,
                               max_len: int = 0) -> int:
    """Bytes of workspace that prefix_attention needs for these arguments (0: it refuses them)."""
    w = kv.view
    with _On(kv.k.device, None):
        return _workspace_bytes(w.n_pages, w.n_seqs, w.max_pages, w.n_kv_heads, w.head_dim, w.elem, n_q_heads, B, T,
                                n_groups, max_prefix, max_len, kv.k.device.index)


def prefix_attention(kv: PagedKV, q: torch.Tensor, group_off: Optional[torch.Tensor] = None,
                     prefix_seq: Optional[torch.Tensor] = None, n_rows: Optional[torch.Tensor] = None, *,
                     seq: Optional[torch.Tensor] = None, causal: bool = True, scale: float = 0.0, max_prefix: int = 0,
                     max_len: int = 0, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """softmax(scale q k^T) v of q [B, T, n_q_heads, head_dim] over the prefix
    of each entry's group (entries group_off[g] .. group_off[g+1] - 1 share the
    cache's sequence prefix_seq[g], -1 for none) and its own sequence seq[b];
    row i of n_rows[b] sees its own tokens j <= length - n_rows[b] + i if
    causal, else all.  Returns out [B, T, n_q_heads, head_dim]; fills lse
    (fp32 [B, T, n_q_heads]) if given."""
    _need(q.dim() == 4 and q.dtype == kv.k.dtype, "q: [B, T, n_q_heads, head_dim] of the cache's type")
    B, T, Hq, dh = q.shape
    dev = kv.k.device
    _need(dh == kv.k.shape[3] and q.device == dev, "q does not have the cache's head_dim or device")
    NG = 0
    if group_off is not None or prefix_seq is not None:
        _need(group_off is not None and prefix_seq is not None, "group_off and prefix_seq come together")
        NG = prefix_seq.numel()
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty((B, T, Hq, dh), dtype=q.dtype, device=dev)
        _need(out.shape == q.shape and out.dtype == q.dtype and out.is_contiguous() and out.device == dev,
              "out: contiguous, the shape and type of q")
        if lse is not None:
            _need(lse.shape == (B, T, Hq) and lse.dtype == torch.float32 and lse.is_contiguous() and lse.device == dev,
                  "lse: contiguous fp32 [B, T, n_q_heads]")
        if workspace is None:
            w = kv.view
            workspace = torch.empty(
                _workspace_bytes(w.n_pages, w.n_seqs, w.max_pages, w.n_kv_heads, w.head_dim, w.elem, Hq, B, T, NG,
                                 max_prefix, max_len, dev.index) or 256, dtype=torch.uint8, device=dev)
        _need(workspace.device == dev and workspace.is_contiguous(), "workspace: contiguous, on the cache's device")
        _lib.check(_lib.lib().dflash_prefix_attention(
            kv.ref, q.data_ptr(), _token_stride(q, "q"), Hq, _ints(n_rows, B, dev, "n_rows"),
            _ints(seq, B, dev, "seq"), B, T, _ints(group_off, NG + 1, dev, "group_off") if NG else None,
            _ints(prefix_seq, NG, dev, "prefix_seq") if NG else None, NG, 1 if causal else 0, scale, max_prefix,
            max_len, out.data_ptr(), None if lse is None else lse.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _status(status, dev), s), "dflash_prefix_attention")
    return out


def gemm_w4(W: torch.Tensor, scale: torch.Tensor, X: torch.Tensor, zero: Optional[torch.Tensor] = None, *,
            group: int, fmt: str = "int4", out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
            stream=None) -> torch.Tensor:
    """X [M, K] (bf16 or fp16, M <= 32) times the transpose of the 4-bit matrix
    W (uint8 [N, K / 2], element 2j in the low half of byte j) under group
    scales [N, ceil(K / group)]: fmt "int4" (code - zero, zero uint8 like the
    scales or None for 8) or "e2m1".  Returns fp32 [M, N]."""
    _need(W.dim() == 2 and W.dtype == torch.uint8 and W.is_contiguous(), "W: contiguous uint8 [N, K / 2]")
    N, K = W.shape[0], W.shape[1] * 2
    dev = W.device
    _need(X.dim() == 2 and X.shape[1] == K and X.is_contiguous() and X.dtype in (torch.bfloat16, torch.float16)
          and X.device == dev, "X: contiguous bf16 or fp16 [M, K] on the device of W")
    _need(fmt in _W4, "fmt: int4 or e2m1")
    M = X.shape[0]
    _need(group > 0, "group: 32, 64 or 128")
    gs = (N, -(-K // group))
    _need(scale.shape == gs and scale.dtype in _ELEM and scale.is_contiguous() and scale.device == dev,
          "scale: contiguous fp32, bf16 or fp16 [N, ceil(K / group)] on the device of W")
    if zero is not None:
        _need(zero.shape == gs and zero.dtype == torch.uint8 and zero.is_contiguous() and zero.device == dev,
              "zero: contiguous uint8 [N, ceil(K / group)] on the device of W")
    with _On(dev, stream) as s:
        if out is None:
            out = torch.empty((M, N), dtype=torch.float32, device=dev)
        _need(out.shape == (M, N) and out.dtype == torch.float32 and out.is_contiguous() and out.device == dev,
              "out: contiguous fp32 [M, N] on the device of W")
        _lib.check(_lib.lib().dflash_gemm_w4(
            W.data_ptr(), _W4[fmt], scale.data_ptr(), _ELEM[scale.dtype], None if zero is None else zero.data_ptr(),
            N, K, group, X.data_ptr(), _ELEM[X.dtype], M, out.data_ptr(), _status(status, dev), s), "dflash_gemm_w4")
    return out
