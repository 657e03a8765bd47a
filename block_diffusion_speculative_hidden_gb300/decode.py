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


_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8
# (the current stream's address and the current device by their own names in
# torch._C: torch.cuda.current_stream() builds an object, 3 us of a 10 us call)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _need(cond, what: str) -> None:
    if not cond:
        raise ValueError(what)


def _on(dev: int, stream: Optional[torch.cuda.Stream]):
    """A guard that makes device `dev` (and `stream`, where given) the current ones, or None where they are."""
    _need(dev >= 0, "tensors must be on a CUDA device")
    if stream is not None:
        _need(stream.device.index == dev, "the stream belongs to another device than the tensors")
        return torch.cuda.stream(stream)
    return None if _current_device() == dev else torch.cuda.device(dev)


def _ints(t: Optional[torch.Tensor], n: int, dev: int, what: str) -> Optional[int]:
    """The address of an optional int32 tensor of n entries."""
    if t is None:
        return None
    if t.dtype is not _I32 or t.numel() != n or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(what + ": contiguous int32 of %d entries on the cache's device" % n)
    return t.data_ptr()


def _token_stride(t: torch.Tensor, what: str) -> int:
    """Elements between tokens of [B, T, heads, head_dim] with contiguous heads and evenly spaced tokens."""
    B, T, H, dh = t.shape
    sb, st, sh, sd = t.stride()
    if sd != 1 or (sh != dh and H != 1):
        raise ValueError(what + ": the heads of a token must be contiguous")
    if T == 1:
        return sb if B > 1 else H * dh
    if B != 1 and sb != T * st:
        raise ValueError(what + ": tokens must be evenly spaced")
    return st


class PagedKV:
    """One layer of a paged KV cache in the caller's tensors: k, v
    [n_pages, n_kv_heads, 16, head_dim] (fp32, bf16 or fp16), page_table int32
    [n_seqs, max_pages], seq_len int32 [n_seqs]."""

    __slots__ = ("k", "v", "page_table", "seq_len", "dev", "shape", "view", "ref")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, seq_len: torch.Tensor):
        n, h, page, dh = k.shape
        rows, most = page_table.shape
        dev, dt = k.get_device(), k.dtype
        _need(page == 16 and v.shape == k.shape, "k, v: [n_pages, n_kv_heads, 16, head_dim]")
        _need(dt in _ELEM and v.dtype is dt, "k, v: fp32, bf16 or fp16, both alike")
        _need(k.is_contiguous() and v.is_contiguous(), "k, v must be contiguous")
        _need(page_table.dtype is _I32 and page_table.is_contiguous(),
              "page_table: contiguous int32 [n_seqs, max_pages]")
        _need(seq_len.dtype is _I32 and seq_len.is_contiguous() and seq_len.numel() == rows,
              "seq_len: contiguous int32 [n_seqs]")
        _need(v.get_device() == dev and page_table.get_device() == dev and seq_len.get_device() == dev,
              "one device for the whole cache")
        self.k, self.v, self.page_table, self.seq_len, self.dev = k, v, page_table, seq_len, dev
        self.shape = (n, rows, most, h, dh, _ELEM[dt])
        self.view = _lib.DflashPagedKV(k.data_ptr(), v.data_ptr(), page_table.data_ptr(), seq_len.data_ptr(),
                                       *self.shape)
        self.ref = ctypes.byref(self.view)


def rope_table(rows: int, head_dim: int, theta: float, device="cuda", stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(cos, sin) fp32 [rows, head_dim / 2] of pos * theta^(-2i / head_dim)."""
    dev = torch.device(device)
    index = _current_device() if dev.index is None else dev.index
    _need(dev.type == "cuda", "the table is made on a CUDA device")
    guard = _on(index, stream)
    if guard is not None:
        with guard:
            return rope_table(rows, head_dim, theta, device=torch.device("cuda", index))
    cos, sin = (torch.empty((rows, head_dim // 2), dtype=_F32, device="cuda") for _ in range(2))
    _lib.check(_lib.lib().dflash_rope_table(cos.data_ptr(), sin.data_ptr(), rows, head_dim, float(theta),
                                            _raw_stream(index)), "dflash_rope_table")
    return cos, sin


def append_kv(kv: PagedKV, k: torch.Tensor, v: torch.Tensor, n_rows: Optional[torch.Tensor] = None, *,
              seq: Optional[torch.Tensor] = None, pos_base: Optional[torch.Tensor] = None,
              rope: Optional[Tuple[torch.Tensor, torch.Tensor]] = None, q: Optional[torch.Tensor] = None,
              q_out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """The rows k, v [B, T, n_kv_heads, head_dim] as the last n_rows[b] tokens
    of sequence seq[b] (whose seq_len already counts them), keys rotated by
    `rope` = (cos, sin) at pos_base[b] + slot; q [B, T, n_q_heads, head_dim]
    rotated alike into q_out (cache type).  Returns q_out."""
    dev = kv.dev
    guard = _on(dev, stream)
    if guard is not None:
        with guard:
            return append_kv(kv, k, v, n_rows, seq=seq, pos_base=pos_base, rope=rope, q=q, q_out=q_out, status=status)
    B, T, H, dh = k.shape
    src = k.dtype
    _need(v.shape == k.shape and v.dtype is src and src in _ELEM, "k, v: [B, T, n_kv_heads, head_dim] of one type")
    _need((H, dh) == kv.shape[3:5], "k, v do not have the cache's heads")
    _need(k.get_device() == dev and v.get_device() == dev, "k, v are on another device than the cache")
    cos = sin = qp = op = None
    rows = ld_q = Hq = 0
    if rope is not None:
        c, s = rope
        rows, half = c.shape
        _need(half * 2 == dh and s.shape == c.shape and c.dtype is _F32 and s.dtype is _F32 and c.is_contiguous()
              and s.is_contiguous() and c.get_device() == dev and s.get_device() == dev,
              "rope: contiguous fp32 (cos, sin) [rows, head_dim / 2] on the cache's device")
        cos, sin = c.data_ptr(), s.data_ptr()
    if q is not None:
        qB, qT, Hq, qd = q.shape
        _need(qB == B and qT == T and qd == dh and q.dtype is src and q.get_device() == dev,
              "q: [B, T, n_q_heads, head_dim], the type of k, on the cache's device")
        if q_out is None:
            q_out = torch.empty((B, T, Hq, dh), dtype=kv.k.dtype, device=k.device)
        _need(q_out.shape == q.shape and q_out.dtype is kv.k.dtype and q_out.is_contiguous()
              and q_out.get_device() == dev, "q_out: contiguous, the shape of q and the cache's type")
        qp, ld_q, op = q.data_ptr(), _token_stride(q, "q"), q_out.data_ptr()
    else:
        _need(q_out is None, "q_out without q")
    _lib.check(_lib.lib().dflash_append_kv(
        kv.ref, k.data_ptr(), _token_stride(k, "k"), v.data_ptr(), _token_stride(v, "v"), _ELEM[src],
        _ints(n_rows, B, dev, "n_rows"), _ints(seq, B, dev, "seq"), _ints(pos_base, B, dev, "pos_base"), B, T,
        cos, sin, rows, qp, ld_q, Hq, op, _ints(status, 1, dev, "status"), _raw_stream(dev)), "dflash_append_kv")
    return q_out


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(shape, Hq, B, T, NG, max_prefix, max_len, dev):
    view = _lib.DflashPagedKV(256, 256, 256, 256, *shape)
    return _lib.lib().dflash_prefix_attention_workspace(ctypes.byref(view), Hq, B, T, NG, max_prefix, max_len)


def prefix_attention_workspace(kv: PagedKV, n_q_heads: int, B: int, T: int, n_groups: int, max_prefix: int = 0,
                               max_len: int = 0) -> int:
    """Bytes of workspace that prefix_attention needs for these arguments (0: it refuses them)."""
    guard = _on(kv.dev, None)
    if guard is not None:
        with guard:
            return prefix_attention_workspace(kv, n_q_heads, B, T, n_groups, max_prefix, max_len)
    return _workspace_bytes(kv.shape, n_q_heads, B, T, n_groups, max_prefix, max_len, kv.dev)


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
    (fp32 [B, T, n_q_heads]) if given.  A call that is recorded into a graph
    wants out and workspace of the caller's, which live as long as the graph."""
    dev = kv.dev
    guard = _on(dev, stream)
    if guard is not None:
        with guard:
            return prefix_attention(kv, q, group_off, prefix_seq, n_rows, seq=seq, causal=causal, scale=scale,
                                    max_prefix=max_prefix, max_len=max_len, out=out, lse=lse, workspace=workspace,
                                    status=status)
    B, T, Hq, dh = q.shape
    dt = q.dtype
    _need(dt is kv.k.dtype and dh == kv.shape[4] and q.get_device() == dev,
          "q: [B, T, n_q_heads, head_dim] of the cache's type, head_dim and device")
    NG = off = pre = 0
    if group_off is not None or prefix_seq is not None:
        _need(group_off is not None and prefix_seq is not None, "group_off and prefix_seq come together")
        NG = prefix_seq.numel()
        off, pre = _ints(group_off, NG + 1, dev, "group_off"), _ints(prefix_seq, NG, dev, "prefix_seq")
    if out is None:
        out = torch.empty((B, T, Hq, dh), dtype=dt, device=q.device)
    elif out.shape != q.shape or out.dtype is not dt or not out.is_contiguous() or out.get_device() != dev:
        raise ValueError("out: contiguous, the shape and type of q")
    lp = None
    if lse is not None:
        _need(lse.shape == (B, T, Hq) and lse.dtype is _F32 and lse.is_contiguous() and lse.get_device() == dev,
              "lse: contiguous fp32 [B, T, n_q_heads]")
        lp = lse.data_ptr()
    if workspace is None:
        size = _workspace_bytes(kv.shape, Hq, B, T, NG, max_prefix, max_len, dev)
        workspace = torch.empty(size or 256, dtype=_U8, device=q.device)
    else:
        _need(workspace.get_device() == dev and workspace.is_contiguous(), "workspace: contiguous, the cache's device")
        size = workspace.numel() * workspace.element_size()
    _lib.check(_lib.lib().dflash_prefix_attention(
        kv.ref, q.data_ptr(), _token_stride(q, "q"), Hq, _ints(n_rows, B, dev, "n_rows"), _ints(seq, B, dev, "seq"), B,
        T, off or None, pre or None, NG, 1 if causal else 0, scale, max_prefix, max_len, out.data_ptr(), lp,
        workspace.data_ptr(), size, _ints(status, 1, dev, "status"), _raw_stream(dev)), "dflash_prefix_attention")
    return out


def gemm_w4(W: torch.Tensor, scale: torch.Tensor, X: torch.Tensor, zero: Optional[torch.Tensor] = None, *,
            group: int, fmt: str = "int4", out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
            stream=None) -> torch.Tensor:
    """X [M, K] (bf16 or fp16, M <= 32) times the transpose of the 4-bit matrix
    W (uint8 [N, K / 2], element 2j in the low half of byte j) under group
    scales [N, ceil(K / group)]: fmt "int4" (code - zero, zero uint8 like the
    scales or None for 8) or "e2m1".  Returns fp32 [M, N]."""
    dev = W.get_device()
    guard = _on(dev, stream)
    if guard is not None:
        with guard:
            return gemm_w4(W, scale, X, zero, group=group, fmt=fmt, out=out, status=status)
    N, K = W.shape
    M, xk = X.shape
    K *= 2
    _need(W.dtype is _U8 and W.is_contiguous(), "W: contiguous uint8 [N, K / 2]")
    _need(xk == K and X.dtype in _ELEM and X.dtype is not _F32 and X.is_contiguous() and X.get_device() == dev,
          "X: contiguous bf16 or fp16 [M, K] on the device of W")
    _need(fmt in _W4, "fmt: int4 or e2m1")
    _need(group > 0, "group: 32, 64 or 128")
    groups = (K + group - 1) // group
    _need(scale.shape == (N, groups) and scale.dtype in _ELEM and scale.is_contiguous() and scale.get_device() == dev,
          "scale: contiguous fp32, bf16 or fp16 [N, ceil(K / group)] on the device of W")
    zp = None
    if zero is not None:
        _need(zero.shape == (N, groups) and zero.dtype is _U8 and zero.is_contiguous() and zero.get_device() == dev,
              "zero: contiguous uint8 [N, ceil(K / group)] on the device of W")
        zp = zero.data_ptr()
    if out is None:
        out = torch.empty((M, N), dtype=_F32, device=W.device)
    elif out.shape != (M, N) or out.dtype is not _F32 or not out.is_contiguous() or out.get_device() != dev:
        raise ValueError("out: contiguous fp32 [M, N] on the device of W")
    _lib.check(_lib.lib().dflash_gemm_w4(
        W.data_ptr(), _W4[fmt], scale.data_ptr(), _ELEM[scale.dtype], zp, N, K, group, X.data_ptr(), _ELEM[X.dtype], M,
        out.data_ptr(), _ints(status, 1, dev, "status"), _raw_stream(dev)), "dflash_gemm_w4")
    return out
