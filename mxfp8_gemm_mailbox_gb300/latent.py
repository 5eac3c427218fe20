"""Latent attention in its absorbed form, the step before the projection.

Thin bindings over the C ABI, as in :mod:`.api`: ``latent_query`` multiplies
the queries into the latent space, ``LatentAttention`` attends over the paged
cache of latents, ``latent_values`` multiplies each head's result by its value
matrix and rounds it to MXFP8, the activations ``PublishGemm`` takes.

A decode step makes these calls once a layer, and the smallest take a few
microseconds on the GPU, so the checks here stay cheap: a dtype, a shape, the
device and the strides of each tensor.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import LatentDesc, check
from .api import _ptr, _stream

_BF16, _I32, _I64 = torch.bfloat16, torch.int32, torch.int64
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
_ROPE = _lib.LATENT_ROPE


def _device_of(t: torch.Tensor, name: str) -> int:
    """The ordinal of t's device, which must be the current CUDA device."""
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if device != torch.cuda.current_device():
        raise ValueError(f"{name} is on device {device}, the current device is "
                         f"{torch.cuda.current_device()}")
    return device


def _expect(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: int) -> None:
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype)[6:]}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor on device {device}")


def _matrices(w: torch.Tensor) -> tuple:
    """The shape of a matrix a head, and its device."""
    if w.dtype is not _BF16:
        raise TypeError(f"w must be bfloat16, got {w.dtype}")
    if w.dim() != 3:
        raise ValueError(f"w must be [heads][outputs][inputs], got {list(w.shape)}")
    device = _device_of(w, "w")
    if not w.is_contiguous():
        raise ValueError("w must be a contiguous CUDA tensor")
    return (*w.shape, device)


def latent_query(q_nope: torch.Tensor, q_rope: torch.Tensor, w: torch.Tensor,
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q [rows][heads][latent + 64]: ``w [heads][latent][nope]`` times
    ``q_nope [rows][heads][nope]``, with ``q_rope [rows][heads][64]`` (already
    rotated) behind it.  ``w[h]`` is head h's key matrix, the latent axis
    first.  ``w`` is read before the kernel before this one on the stream has
    finished, so that kernel must not write it."""
    heads, latent, nope, device = _matrices(w)
    rows = len(q_nope)
    _expect(q_nope, "q_nope", _BF16, (rows, heads, nope), device)
    _expect(q_rope, "q_rope", _BF16, (rows, heads, _ROPE), device)
    if out is None:
        out = w.new_empty((rows, heads, latent + _ROPE))
    else:
        _expect(out, "out", _BF16, (rows, heads, latent + _ROPE), device)
    status = _lib.load().mxfp8_latent_query(q_nope.data_ptr(), q_rope.data_ptr(), w.data_ptr(),
                                            out.data_ptr(), rows, heads, nope, latent,
                                            _stream(stream))
    if status:
        check(status, "mxfp8_latent_query")
    return out


def _codes_out(t: torch.Tensor, name: str, rows: int, cols: int, device: int) -> None:
    if t.element_size() != 1:
        raise TypeError(f"{name} must hold one-byte codes (uint8 / float8), got {t.dtype}")
    _expect(t, name, t.dtype, (rows, cols), device)


def latent_values(o: torch.Tensor, w: torch.Tensor, x: torch.Tensor | None = None,
                  x_scale: torch.Tensor | None = None, stream=None):
    """(x, x_scale): ``w [heads][value][latent]`` times ``o [rows][heads][latent]``
    in MXFP8, E4M3 elements ``[rows][heads * value]`` and E8M0 scales
    ``[rows][heads * value / 32]``, which ``PublishGemm.run`` takes.  ``w`` is
    read before the kernel before this one on the stream has finished, so that
    kernel must not write it."""
    heads, value, latent, device = _matrices(w)
    rows, k = len(o), heads * value
    _expect(o, "o", _BF16, (rows, heads, latent), device)
    if x is None:
        x = w.new_empty((rows, k), dtype=_E4M3)
    else:
        _codes_out(x, "x", rows, k, device)
    if x_scale is None:
        x_scale = w.new_empty((rows, k // 32), dtype=_E8M0)
    else:
        _codes_out(x_scale, "x_scale", rows, k // 32, device)
    status = _lib.load().mxfp8_latent_values(o.data_ptr(), w.data_ptr(), x.data_ptr(),
                                             x_scale.data_ptr(), rows, heads, latent, value,
                                             _stream(stream))
    if status:
        check(status, "mxfp8_latent_values")
    return x, x_scale


class LatentAttention:
    """Attention of ``heads`` query heads over a paged cache of latents.

    Holds the workspace and the flags word, so calls on one object are ordered
    on one stream and made by one host thread at a time."""

    def __init__(self, heads: int, latent: int = 512, device=None):
        nbytes = _lib.load().mxfp8_latent_workspace_bytes(latent)
        if nbytes == 0:
            raise ValueError(f"latent must be 256 or 512, got {latent}")
        device = torch.device(device or "cuda")
        self.heads, self.latent = heads, latent
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.flags = torch.zeros(1, dtype=torch.int32, device=device)
        self._desc = LatentDesc(heads, latent)
        self._borrowed = (ctypes.byref(self._desc), self.workspace.data_ptr(), nbytes)

    def run(self, q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor,
            lengths: torch.Tensor, row_begin: torch.Tensor, scale: float,
            tree: torch.Tensor | None = None, out: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
        """out [rows][heads][latent] of ``q [rows][heads][latent + 64]`` over
        ``cache [pages][page_size][latent + 64]`` (pages and tokens may be
        strided).  ``page_table`` int32 [requests][width], ``lengths`` int32
        [requests] (the drafts' latents included), ``row_begin`` int32
        [requests + 1]: request b's drafts are rows ``row_begin[b]`` to
        ``row_begin[b + 1] - 1`` of q and the last tokens of its cache.  Every
        row sees the tokens before the drafts; of the drafts, row t sees j iff
        bit j of ``tree[t]`` (int64 [rows], j < 64) is set, without a tree iff
        j <= t."""
        heads, latent = self.heads, self.latent
        width = latent + _ROPE
        if q.dim() != 3:
            raise ValueError(f"q must be [rows][{heads}][{width}], got {list(q.shape)}")
        rows = len(q)
        if q.shape != (rows, heads, width):
            raise ValueError(f"q must be [rows][{heads}][{width}], got {list(q.shape)}")
        device = _device_of(q, "q")
        _expect(q, "q", _BF16, (rows, heads, width), device)
        if cache.dtype is not _BF16:
            raise TypeError(f"cache must be bfloat16, got {cache.dtype}")
        shape = cache.shape
        if len(shape) != 3 or shape[2] != width:
            raise ValueError(f"cache must be [pages][page_size][{width}], got {list(shape)}")
        page_stride, token_stride, one = cache.stride()
        if cache.get_device() != device or one != 1:
            raise ValueError(f"cache must be a CUDA tensor on device {device} with contiguous "
                             "tokens")
        if lengths.dim() != 1 or page_table.dim() != 2:
            raise ValueError("lengths must be [requests] and page_table [requests][width], got "
                             f"{list(lengths.shape)} and {list(page_table.shape)}")
        requests, table_width = page_table.shape
        _expect(lengths, "lengths", _I32, (requests,), device)
        _expect(row_begin, "row_begin", _I32, (requests + 1,), device)
        _expect(page_table, "page_table", _I32, (requests, table_width), device)
        if tree is not None:
            _expect(tree, "tree", _I64, (rows,), device)
        if out is None:
            out = q.new_empty((rows, heads, latent))
        else:
            _expect(out, "out", _BF16, (rows, heads, latent), device)
        d = self._desc
        d.rows, d.requests, d.page_size, d.pages = rows, requests, shape[1], shape[0]
        d.table_width, d.scale, d.token_stride, d.page_stride = (table_width, scale, token_stride,
                                                                 page_stride)
        desc, workspace, nbytes = self._borrowed
        status = _lib.load().mxfp8_latent_attend(
            desc, q.data_ptr(), cache.data_ptr(), page_table.data_ptr(), lengths.data_ptr(),
            row_begin.data_ptr(), _ptr(tree), out.data_ptr(), workspace, nbytes,
            self.flags.data_ptr(), _stream(stream))
        if status:
            check(status, "mxfp8_latent_attend")
        return out

    def status(self, stream=None) -> int:
        """The FLAG_* bits raised so far; synchronises the stream."""
        from .api import _synchronize

        _synchronize(stream, self.flags.device)
        return int(self.flags.item())
