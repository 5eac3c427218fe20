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
from .api import _current_device, _stream

_BF16, _I32, _I64 = torch.bfloat16, torch.int32, torch.int64
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
_ROPE = _lib.LATENT_ROPE
_empty = torch.empty


def _refuse(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: int) -> None:
    """Raises what is wrong with a tensor that is not dtype, shape, contiguous
    and on the device."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {str(dtype)[6:]}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if device < 0 or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor on device {max(device, 0)}")


def _expect(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device: int) -> None:
    if (t.dtype is not dtype or t.shape != shape or t.get_device() != device
            or not t.is_contiguous()):
        _refuse(t, name, dtype, shape, device)


def _check_device(device: int, name: str) -> None:
    if device < 0:
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if device != _current_device():
        raise ValueError(f"{name} is on device {device}, the current device is "
                         f"{_current_device()}")


def _matrices(w: torch.Tensor) -> tuple:
    """The shape of a matrix a head, and its device."""
    if w.dtype is not _BF16:
        raise TypeError(f"w must be bfloat16, got {w.dtype}")
    if w.dim() != 3:
        raise ValueError(f"w must be [heads][outputs][inputs], got {list(w.shape)}")
    device = w.get_device()
    _check_device(device, "w")
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
    rows = q_nope.shape[0]
    _expect(q_nope, "q_nope", _BF16, (rows, heads, nope), device)
    _expect(q_rope, "q_rope", _BF16, (rows, heads, _ROPE), device)
    if out is None:
        out = _empty((rows, heads, latent + _ROPE), dtype=_BF16, device=w.device)
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
    rows, k = o.shape[0], heads * value
    _expect(o, "o", _BF16, (rows, heads, latent), device)
    if x is None:
        x = _empty((rows, k), dtype=_E4M3, device=w.device)
    else:
        _codes_out(x, "x", rows, k, device)
    if x_scale is None:
        x_scale = _empty((rows, k // 32), dtype=_E8M0, device=w.device)
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
        self._borrowed = (ctypes.byref(self._desc), self.workspace.data_ptr(), nbytes,
                          self.flags.data_ptr())

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
        shape = q.shape
        if len(shape) != 3 or shape[1] != heads or shape[2] != width:
            raise ValueError(f"q must be [rows][{heads}][{width}], got {list(shape)}")
        rows, device = shape[0], q.get_device()
        _check_device(device, "q")
        if q.dtype is not _BF16 or not q.is_contiguous():
            _refuse(q, "q", _BF16, shape, device)
        if cache.dtype is not _BF16:
            raise TypeError(f"cache must be bfloat16, got {cache.dtype}")
        pool = cache.shape
        if len(pool) != 3 or pool[2] != width:
            raise ValueError(f"cache must be [pages][page_size][{width}], got {list(pool)}")
        page_stride, token_stride, one = cache.stride()
        if cache.get_device() != device or one != 1:
            raise ValueError(f"cache must be a CUDA tensor on device {device} with contiguous "
                             "tokens")
        table = page_table.shape
        if len(table) != 2:
            raise ValueError(f"page_table must be [requests][width], got {list(table)}")
        requests = table[0]
        _expect(page_table, "page_table", _I32, table, device)
        _expect(lengths, "lengths", _I32, (requests,), device)
        _expect(row_begin, "row_begin", _I32, (requests + 1,), device)
        masks = None
        if tree is not None:
            _expect(tree, "tree", _I64, (rows,), device)
            masks = tree.data_ptr()
        if out is None:
            out = _empty((rows, heads, latent), dtype=_BF16, device=q.device)
        else:
            _expect(out, "out", _BF16, (rows, heads, latent), device)
        d = self._desc
        d.rows = rows
        d.requests = requests
        d.page_size = pool[1]
        d.pages = pool[0]
        d.table_width = table[1]
        d.scale = scale
        d.token_stride = token_stride
        d.page_stride = page_stride
        desc, workspace, nbytes, flags = self._borrowed
        status = _lib.load().mxfp8_latent_attend(
            desc, q.data_ptr(), cache.data_ptr(), page_table.data_ptr(), lengths.data_ptr(),
            row_begin.data_ptr(), masks, out.data_ptr(), workspace, nbytes, flags,
            _stream(stream))
        if status:
            check(status, "mxfp8_latent_attend")
        return out

    def status(self, stream=None) -> int:
        """The FLAG_* bits raised so far; synchronises the stream."""
        from .api import _synchronize

        _synchronize(stream, self.flags.device)
        return int(self.flags.item())
