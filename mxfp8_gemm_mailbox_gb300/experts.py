"""A layer of routed experts in microscaled formats, what follows the projection.

Thin bindings over the C ABI, as in :mod:`.api`: ``route`` chooses each token's
experts and orders the tokens by expert, ``quantize`` rounds their rows to MXFP8
or MXFP4, ``ExpertProduct`` multiplies every expert's matrix by its rows (with a
gate, the first product of a layer; without, the second, or one matrix of a whole
prompt), ``combine`` sums what each token's experts gave.

    routing = route(logits, 8)
    h, h_scale = quantize(x, "mxfp8", rows=routing.row)
    h, h_scale = gate_up.run(h, h_scale, routing.begin, format="mxfp8")
    y = down.run(h, h_scale, routing.begin)
    out = combine(y, routing.weight, routing.slot, add=x)

No step reads anything back, so the layer can be captured into a CUDA graph.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _lib
from ._lib import check


class Routing(NamedTuple):
    """``weight`` FP32 and ``expert`` int32 [tokens][k], ``slot`` int32 [tokens][k]
    (the row of each choice in the experts' products, -1 for none), ``row`` int32
    [tokens * k] (the token of each row, -1 past the last), ``begin`` int32
    [experts + 1] (where each expert's rows begin).  The five lie in one piece of memory
    (with the call's workspace): keeping or saving one keeps or saves all, a ``clone`` of
    it does not."""

    weight: torch.Tensor
    expert: torch.Tensor
    slot: torch.Tensor
    row: torch.Tensor
    begin: torch.Tensor


def route(logits: torch.Tensor, k: int, normalize: bool = True, stream=None) -> Routing:
    """Each token's ``k`` experts of the largest ``logits [tokens][experts]`` (BF16,
    FP16 or FP32; rows may be strided), ties to the lowest index, weighted by
    exp(z - z_max) over the sum of those of the chosen (``normalize``) or of all.
    A logit of -infinity is not chosen (expert and slot -1, weight 0); NaN counts
    as the largest."""
    return Routing(*_lib.calls().route(logits, k, normalize, stream))


def quantize(x: torch.Tensor, format: str, rows: torch.Tensor | None = None,
             codes: torch.Tensor | None = None, scale: torch.Tensor | None = None,
             flags: torch.Tensor | None = None, stream=None):
    """(codes, scale) of ``x [...][K]`` (BF16, FP16 or FP32; the rows of a matrix may be
    strided): ``"mxfp8"`` E4M3 ``[...][K]``, ``"mxfp4"`` E2M1 ``[...][K / 2]`` (uint8, the
    even element in the low half), E8M0 scales ``[...][K / 32]``.  With ``rows`` (int32)
    output row r is made of ``x[rows[r]]``; -1 leaves it as it was, and another index
    outside x too, which raises FLAG_BAD_INDEX in ``flags`` (int32 [1]).  What is not
    finite becomes NaN, in MXFP4 its whole block."""
    return _lib.calls().quantize(x, format, rows, codes, scale, flags, stream)


_TYPES = {torch.bfloat16: _lib.BF16, torch.float16: _lib.FP16, torch.float32: _lib.FP32}


def dequantize(codes: torch.Tensor, scale: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
               stream=None) -> torch.Tensor:
    """The values ``[...][K]`` of codes as ``quantize`` makes them; FP32 holds every value
    below 2^128 (numbers within half a step of it are rounded up to it, and come back
    infinite), BF16 and FP16 (``dtype``) what rounds to them."""
    if dtype not in _TYPES:
        raise TypeError(f"dtype must be bfloat16, float16 or float32, got {dtype}")
    return _lib.calls().dequantize(codes, scale, _TYPES[dtype], stream)


class ExpertProduct:
    """Matrices ``w [experts][N][K]`` (E4M3 codes) or ``[experts][N][K / 2]`` (E2M1) with
    their scales ``w_scale [experts][N][K / 32]``, or one of them without the first axis.
    ``gated``: N holds a gate's rows, then as many of an up matrix, and the result is
    silu(gate) x up, N / 2 wide.

    For matrices that stay: the codes are borrowed and read in place, while the scales are
    copied, once, into the products' order, and the constructor waits for that.  New codes
    written into ``w`` are what the next call reads; for new scales, make another object.
    The workspace (5 MB) and the flags word live here; ``workspace``: another product's, to
    be shared.  Calls that share one are ordered on
    one stream, made by one host thread at a time, and the object outlives what they have
    queued on another stream than the one it was made on."""

    def __init__(self, w: torch.Tensor, w_scale: torch.Tensor, gated: bool = False,
                 workspace: torch.Tensor | None = None):
        from .api import _on_device, _synchronize

        for t, name in ((w, "w"), (w_scale, "w_scale")):
            if t.element_size() != 1:
                raise TypeError(f"{name} must hold one-byte codes (uint8 / float8), got {t.dtype}")
            if t.dim() not in (2, 3):
                raise ValueError(f"{name} must be [experts][N][...] or [N][...], got "
                                 f"{tuple(t.shape)}")
        k = 32 * w_scale.shape[-1]
        if w.shape[:-1] != w_scale.shape[:-1] or w.shape[-1] not in (k, k // 2):
            raise ValueError("w must be [experts][N][K] (E4M3) or [experts][N][K / 2] (E2M1) and "
                             f"w_scale [experts][N][K / 32], got {tuple(w.shape)} and "
                             f"{tuple(w_scale.shape)}")
        outputs = w.shape[-2]
        if gated and outputs % 2:
            raise ValueError(f"gated, N must be even, got {outputs}")
        _on_device(w, "w")
        _on_device(w_scale, "w_scale")
        if w.device != w_scale.device:
            raise ValueError(f"w is on {w.device}, w_scale on {w_scale.device}")
        lib = _lib.load()
        self.experts = w.shape[0] if w.dim() == 3 else 1
        self.n, self.k, self.gated = outputs // 2 if gated else outputs, k, bool(gated)
        w_format = _lib.FORMAT_MXFP8 if w.shape[-1] == k else _lib.FORMAT_MXFP4
        desc = _lib.ExpertDesc(self.experts, self.n, k, self.gated, w_format)
        nbytes = lib.mxfp8_expert_scales_bytes(ctypes.byref(desc))
        if nbytes == 0:
            raise ValueError(lib.mxfp8_last_error().decode())
        need = lib.mxfp8_expert_workspace_bytes()
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=w.device)
            workspace[:_lib.EXPERT_WORKSPACE_ZEROS].zero_()
        elif (workspace.dtype != torch.uint8 or workspace.numel() < need
              or workspace.device != w.device or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be another product's on {w.device}")
        self.w, self.workspace = w, workspace
        self.scales = torch.empty(nbytes, dtype=torch.uint8, device=w.device)
        self.flags = torch.zeros(1, dtype=torch.int32, device=w.device)
        with torch.cuda.device(w.device):
            check(lib.mxfp8_expert_lay_scales(ctypes.byref(desc), w_scale.data_ptr(),
                                              self.scales.data_ptr(),
                                              torch.cuda.current_stream().cuda_stream),
                  "mxfp8_expert_lay_scales")
        _synchronize(None, w.device)
        self._own = (self.experts, self.n, k, int(self.gated), w_format, w, self.scales, workspace,
                     self.flags)

    def run(self, x: torch.Tensor, x_scale: torch.Tensor, begin: torch.Tensor | None = None,
            format: str | None = None, out: torch.Tensor | None = None,
            out_scale: torch.Tensor | None = None, stream=None):
        """Rows ``begin[e] .. begin[e + 1] - 1`` of ``x`` (MXFP8 ``[rows][K]`` or MXFP4
        ``[rows][K / 2]``, ``x_scale [rows][K / 32]``) times expert e's matrix: BF16
        ``[rows][N]``, or with a ``format`` ``(codes, scale)`` as ``quantize`` makes them.
        ``begin``: int32 [experts + 1], read on the device; may be left out with one
        expert.  Rows of no expert are left as they were."""
        return _lib.calls().expert_product(*self._own, x, x_scale, begin, format, out, out_scale,
                                           stream)

    def status(self, stream=None) -> int:
        """The FLAG_* bits raised so far; synchronises the stream."""
        from .api import _synchronize

        _synchronize(stream, self.flags.device)
        return int(self.flags.item())


def combine(y: torch.Tensor, weight: torch.Tensor, slot: torch.Tensor,
            add: torch.Tensor | None = None, out: torch.Tensor | None = None,
            flags: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """BF16 ``[tokens][N]``: ``add[t]`` (if given) plus the sum over j of ``weight[t][j]``
    (FP32) times ``y[slot[t][j]]`` (BF16 rows, may be strided), rounded once.  A slot of -1
    (int32) adds nothing; another one outside y neither, and raises FLAG_BAD_INDEX in
    ``flags`` (int32 [1])."""
    return _lib.calls().combine(y, weight, slot, add, out, flags, stream)
