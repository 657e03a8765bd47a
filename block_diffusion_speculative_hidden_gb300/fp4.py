"""Microscaled 4-bit floats: rows quantised, taken back, and multiplied.  Thin
faces (csrc/faces.cpp) of dflash_quantize_fp4, dflash_dequantize_fp4, dflash_fp4_tile_scales and
dflash_gemm_fp4 (include/dflash.h states the formats, what each computes,
checks and refuses).  Streams and memory as in decode.py.
"""
from __future__ import annotations

from operator import attrgetter
from typing import Optional

import torch

from . import _lib
from .decode import _U8, _need, _on, _raw_stream

_FMT = {"mx": _lib.FP4_MX, "nv": _lib.FP4_NV}
_GROUP = {"mx": 32, "nv": 16}
_faces = _lib.faces


def _scale_bytes(rows: int, cols: int, fmt: str) -> int:
    """Bytes of the scale tiles of a [rows, cols] matrix."""
    return -(-rows // 128) * -(-cols // 256) * (2048 if fmt == "nv" else 1024)


class Fp4:
    """A matrix [rows, cols] of microscaled 4-bit floats: codes uint8
    [rows, cols / 2], scales uint8 (tiles of 128 rows x 4 groups, any shape),
    fmt "mx" (a power of two for 32 neighbours) or "nv" (an E4M3 number for 16,
    times the tensor's own `scale`, fp32 of one entry or None for 1).  The
    tensors' addresses are taken once: they cannot be replaced by others."""

    __slots__ = ("_m",)

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, fmt: str, scale: Optional[torch.Tensor] = None):
        self._m = _faces.matrix(codes, scales, fmt, scale)

    @staticmethod
    def _of(m) -> "Fp4":
        t = object.__new__(Fp4)
        t._m = m
        return t

    @staticmethod
    def _empty(rows: int, cols: int, fmt: str, scale: Optional[torch.Tensor], dev: int, device) -> "Fp4":
        """Room for a matrix, in one piece of memory."""
        return Fp4._of(_faces.matrix_room(rows, cols, fmt, scale, torch.empty(0, device=device)))

    codes, scales, scale, rows, cols, fmt, dev, at = (
        property(attrgetter("_m." + _n)) for _n in ("codes", "scales", "scale", "rows", "cols", "fmt", "dev", "at"))

    @property
    def device(self) -> torch.device:
        return self.codes.device

    def __reduce__(self):
        """Copies and pickles are matrices of copied tensors, with addresses of their own."""
        return Fp4, (self.codes, self.scales, self.fmt, self.scale)

    @staticmethod
    def from_rows(codes: torch.Tensor, scales: torch.Tensor, fmt: str, scale: Optional[torch.Tensor] = None,
                  stream=None) -> "Fp4":
        """Of row-major scales uint8 [rows, cols / 32 (mx) or 16 (nv)], as checkpoints hold them."""
        dev = codes.get_device()
        guard = _on(dev, stream)
        if guard is not None:
            with guard:
                return Fp4.from_rows(codes, scales, fmt, scale)
        _need(fmt in _FMT, "fmt: mx or nv")
        _need(codes.dim() == 2 and codes.dtype is _U8, "codes: contiguous uint8 [rows, cols / 2]")
        rows, cols = codes.shape[0], 2 * codes.shape[1]
        _need(cols % 32 == 0, "cols: a multiple of 32")
        _need(scales.shape == (rows, cols // _GROUP[fmt]) and scales.dtype is _U8 and scales.is_contiguous()
              and scales.get_device() == dev, "scales: contiguous uint8 [rows, cols / group] on the codes' device")
        tiles = torch.empty(_scale_bytes(rows, cols, fmt), dtype=_U8, device=codes.device)
        out = Fp4(codes, tiles, fmt, scale)
        _lib.check(_lib.lib().dflash_fp4_tile_scales(scales.data_ptr(), _FMT[fmt], rows, cols, tiles.data_ptr(),
                                                     _raw_stream(dev)), "dflash_fp4_tile_scales")
        return out


def quantize_fp4(x: torch.Tensor, fmt: str = "mx", *, scale: Optional[torch.Tensor] = None, out: Optional[Fp4] = None,
                 stream=None) -> Fp4:
    """x [rows, cols] (fp32, bf16 or fp16; rows may be apart) as microscaled
    4-bit floats; scale (nv): the tensor's number, e.g. its largest magnitude /
    (448 * 6), which `out` then has in place of the one before."""
    if stream is not None:
        with _on(x.get_device(), stream):
            return quantize_fp4(x, fmt, scale=scale, out=out)
    m = _faces.quantize(x, fmt, scale, None if out is None else out._m)
    return Fp4._of(m) if out is None else out


def dequantize_fp4(t: Fp4, dtype: torch.dtype = torch.bfloat16, *, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """The values of t, [rows, cols] of dtype."""
    if stream is not None:
        with _on(t.dev, stream):
            return dequantize_fp4(t, dtype, out=out)
    return _faces.dequantize(t._m, dtype, out)


def gemm_fp4(W: Fp4, X: Fp4, *, dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
             status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """X [M, K] times the transpose of W [N, K], both of one format: [M, N] of
    dtype (bf16, fp16 or fp32), summed in fp32."""
    if stream is not None:
        with _on(W.dev, stream):
            return gemm_fp4(W, X, dtype=dtype, out=out, status=status)
    return _faces.gemm(W._m, X._m, dtype, out, status)
