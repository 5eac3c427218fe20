"""Latent attention in its absorbed form, the step before the projection.

Thin bindings over the C ABI, as in :mod:`.api`: ``latent_query`` multiplies
the queries into the latent space, ``LatentAttention`` attends over the paged
cache of latents, ``latent_values`` multiplies each head's result by its value
matrix and rounds it to MXFP8, the activations ``PublishGemm`` takes.

A decode step makes these calls once a layer, and the smallest take a few
microseconds on the GPU, so their checks and outputs are made in the module
``_calls``.  The products are made for the projection's few rows: they read
their matrices again for every 8 of them.
"""
from __future__ import annotations

import torch

from . import _lib


def latent_query(q_nope: torch.Tensor, q_rope: torch.Tensor, w: torch.Tensor,
                 out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q [rows][heads][latent + 64]: ``w [heads][latent][nope]`` times
    ``q_nope [rows][heads][nope]``, with ``q_rope [rows][heads][64]`` (already
    rotated) behind it.  ``w[h]`` is head h's key matrix, the latent axis
    first.  ``w`` is read before the kernel before this one on the stream has
    finished, so that kernel must not write it."""
    return _lib.calls().latent_query(q_nope, q_rope, w, out, stream)


def latent_values(o: torch.Tensor, w: torch.Tensor, x: torch.Tensor | None = None,
                  x_scale: torch.Tensor | None = None, stream=None):
    """(x, x_scale): ``w [heads][value][latent]`` times ``o [rows][heads][latent]``
    in MXFP8, E4M3 elements ``[rows][heads * value]`` and E8M0 scales
    ``[rows][heads * value / 32]``, which ``PublishGemm.run`` takes.  What is
    not finite becomes NaN.  ``w`` is read before the kernel before this one on
    the stream has finished, so that kernel must not write it."""
    return _lib.calls().latent_values(o, w, x, x_scale, stream)


class LatentAttention:
    """Attention of ``heads`` query heads over a paged cache of latents.

    Holds the workspace (42 MB at latent 512, 21 MB at 256) and the flags word,
    so calls on one object are ordered on one stream and made by one host thread
    at a time, and the object outlives what they have queued on another stream
    than the one it was made on.  One object serves every layer of a stream."""

    def __init__(self, heads: int, latent: int = 512, device=None):
        nbytes = _lib.load().mxfp8_latent_workspace_bytes(latent)
        if nbytes == 0:
            raise ValueError(f"latent must be 256 or 512, got {latent}")
        device = torch.device(device or "cuda")
        self.heads, self.latent = heads, latent
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.flags = torch.zeros(1, dtype=torch.int32, device=device)
        self._own = (heads, latent, self.workspace, nbytes, self.flags)

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
        return _lib.calls().latent_attend(*self._own, q, cache, page_table, lengths, row_begin,
                                          scale, tree, out, stream)

    def status(self, stream=None) -> int:
        """The FLAG_* bits raised so far; synchronises the stream."""
        from .api import _synchronize

        _synchronize(stream, self.flags.device)
        return int(self.flags.item())
