"""Latent attention in its absorbed form, the step before the projection.

Thin bindings over the C ABI, as in :mod:`.api`: ``latent_query`` multiplies
the queries into the latent space, ``LatentAttention`` attends over the paged
cache of latents, ``latent_values`` multiplies each head's result by its value
matrix and rounds it to MXFP8, the activations ``PublishGemm`` takes.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import LatentDesc, check
from .api import _on_device, _ptr, _stream


def _bf16(t: torch.Tensor, name: str, *shape) -> None:
    """Checks a contiguous BF16 tensor; None in ``shape`` is any size."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if t.dim() != len(shape) or any(s is not None and s != d for s, d in zip(shape, t.shape)):
        want = "".join(f"[{'any' if s is None else s}]" for s in shape)
        raise ValueError(f"{name} must be {want}, got {tuple(t.shape)}")
    _on_device(t, name)


def _ints(t: torch.Tensor, name: str, dtype, *shape) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {tuple(t.shape)}")
    _on_device(t, name)


def latent_query(q_nope: torch.Tensor, q_rope: torch.Tensor, w: torch.Tensor,
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q [rows][heads][latent + 64]: ``w [heads][latent][nope]`` times
    ``q_nope [rows][heads][nope]``, with ``q_rope [rows][heads][64]`` (already
    rotated) behind it.  ``w[h]`` is head h's key matrix, the latent axis
    first."""
    _bf16(w, "w", None, None, None)
    heads, latent, nope = w.shape
    _bf16(q_nope, "q_nope", None, heads, nope)
    rows = q_nope.shape[0]
    _bf16(q_rope, "q_rope", rows, heads, _lib.LATENT_ROPE)
    width = latent + _lib.LATENT_ROPE
    if out is None:
        out = torch.empty((rows, heads, width), dtype=torch.bfloat16, device=w.device)
    else:
        _bf16(out, "out", rows, heads, width)
    check(_lib.load().mxfp8_latent_query(_ptr(q_nope), _ptr(q_rope), _ptr(w), _ptr(out), rows,
                                         heads, nope, latent, _stream(stream)),
          "mxfp8_latent_query")
    return out


def latent_values(o: torch.Tensor, w: torch.Tensor, x: torch.Tensor | None = None,
                  x_scale: torch.Tensor | None = None, stream=None):
    """(x, x_scale): ``w [heads][value][latent]`` times ``o [rows][heads][latent]``
    in MXFP8, E4M3 elements ``[rows][heads * value]`` and E8M0 scales
    ``[rows][heads * value / 32]``, which ``PublishGemm.run`` takes."""
    _bf16(w, "w", None, None, None)
    heads, value, latent = w.shape
    _bf16(o, "o", None, heads, latent)
    rows, k = o.shape[0], heads * value
    if x is None:
        x = torch.empty((rows, k), dtype=torch.float8_e4m3fn, device=w.device)
    if x_scale is None:
        x_scale = torch.empty((rows, k // 32), dtype=torch.float8_e8m0fnu, device=w.device)
    for t, name, cols in ((x, "x", k), (x_scale, "x_scale", k // 32)):
        if t.element_size() != 1:
            raise TypeError(f"{name} must hold one-byte codes (uint8 / float8), got {t.dtype}")
        if tuple(t.shape) != (rows, cols):
            raise ValueError(f"{name} must be [{rows}][{cols}], got {tuple(t.shape)}")
        _on_device(t, name)
    check(_lib.load().mxfp8_latent_values(_ptr(o), _ptr(w), _ptr(x), _ptr(x_scale), rows, heads,
                                          latent, value, _stream(stream)), "mxfp8_latent_values")
    return x, x_scale


class LatentAttention:
    """Attention of ``heads`` query heads over a paged cache of latents.

    Holds the workspace and the flags word, so calls on one object are ordered
    on one stream."""

    def __init__(self, heads: int, latent: int = 512, device=None):
        nbytes = _lib.load().mxfp8_latent_workspace_bytes(latent)
        if nbytes == 0:
            raise ValueError(f"latent must be 256 or 512, got {latent}")
        device = torch.device(device or "cuda")
        self.heads, self.latent = heads, latent
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.flags = torch.zeros(1, dtype=torch.int32, device=device)

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
        width = self.latent + _lib.LATENT_ROPE
        _bf16(q, "q", None, self.heads, width)
        rows = q.shape[0]
        if cache.dtype != torch.bfloat16:
            raise TypeError(f"cache must be bfloat16, got {cache.dtype}")
        if cache.dim() != 3 or cache.shape[2] != width:
            raise ValueError(f"cache must be [pages][page_size][{width}], got "
                             f"{tuple(cache.shape)}")
        if not cache.is_cuda or cache.stride(2) != 1:
            raise ValueError("cache must be a CUDA tensor with contiguous tokens")
        requests = lengths.shape[0] if lengths.dim() == 1 else -1
        _ints(lengths, "lengths", torch.int32, max(requests, 0))
        _ints(row_begin, "row_begin", torch.int32, requests + 1)
        if page_table.dim() != 2:
            raise ValueError(f"page_table must be [requests][width], got {tuple(page_table.shape)}")
        _ints(page_table, "page_table", torch.int32, requests, page_table.shape[1])
        if tree is not None:
            _ints(tree, "tree", torch.int64, rows)
        if out is None:
            out = torch.empty((rows, self.heads, self.latent), dtype=torch.bfloat16,
                              device=q.device)
        else:
            _bf16(out, "out", rows, self.heads, self.latent)
        desc = LatentDesc(self.heads, self.latent, rows, requests, cache.shape[1],
                          cache.shape[0], page_table.shape[1], scale, cache.stride(1),
                          cache.stride(0))
        check(_lib.load().mxfp8_latent_attend(
            ctypes.byref(desc), _ptr(q), _ptr(cache), _ptr(page_table), _ptr(lengths),
            _ptr(row_begin), _ptr(tree), _ptr(out), _ptr(self.workspace), self.workspace.nbytes,
            _ptr(self.flags), _stream(stream)), "mxfp8_latent_attend")
        return out

    def status(self, stream=None) -> int:
        """The FLAG_* bits raised so far; synchronises the stream."""
        from .api import _synchronize

        _synchronize(stream, self.flags.device)
        return int(self.flags.item())
