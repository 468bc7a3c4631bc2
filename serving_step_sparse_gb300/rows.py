"""Operators on the cache's FP8 rows: rotary positions, packing, attention, joining.

A row is 656 bytes: 512 e4m3 codes (the latent), 4 fp32 scales (one for each block of
128 channels), 64 bf16 rope channels.  A decode layer packs its new tokens into rows
(``pack``, whose rows go to ``UlaCache.alloc``), turns its queries' rope channels
(``rotate``), attends over the rows that ``UlaCache.step_group`` gathered (``attend``) and
joins partial results over disjoint rows (``join``: ``UlaTP``'s local and remote rows).

Every step runs in the CUDA library through the C ABI (``ula``); this module checks and
marshals arguments.  Calls run on ``stream`` (default: the current stream of the tensors'
device) and return without waiting.  Wrong shapes, types or devices raise ValueError,
errors of the C ABI ``ula.UlaError``.
"""
from __future__ import annotations

import functools

import torch

from . import ula
from .ula import ROPE_PAIRS, ROW_BYTES, ROW_LATENT, ROW_ROPE

_TYPES = {torch.bfloat16: ula.TYPE_BF16, torch.float16: ula.TYPE_F16, torch.float32: ula.TYPE_F32}
_PAIRINGS = {"adjacent": ula.PAIR_ADJACENT, "halves": ula.PAIR_HALVES}


def _on_stream(call):
    """Gives an operator its ``stream`` argument: the call runs (copies and outputs it makes
    included) on that stream, and the tensors handed in, which another stream's allocator may
    own, are recorded there, so that their memory is not handed out again while it runs."""

    @functools.wraps(call)
    def on(*args, stream: torch.cuda.Stream | None = None, **kw):
        if stream is None:
            return call(*args, **kw)
        with torch.cuda.stream(stream):
            result = call(*args, **kw)
        for t in _tensors((args, tuple(kw.values()))):
            t.record_stream(stream)
        return result

    return on


def _tensors(v):
    if isinstance(v, torch.Tensor):
        yield v
    elif isinstance(v, (list, tuple)):
        for x in v:
            yield from _tensors(x)


def _stream_of(*tensors) -> int:
    """The current stream of the tensors' device, which has to be the current device."""
    index = tensors[0].get_device()
    if index < 0 or index != torch.cuda.current_device():
        raise ValueError("the tensors must be on the current CUDA device")
    for t in tensors:
        if t.get_device() != index:
            raise ValueError("the tensors must be on one device")
    return torch._C._cuda_getCurrentRawStream(index)


class Rotary:
    """Rotary positions with one or several axes: pair j of the 64 rope channels is turned by
    ``pos[axis[j]] * freq[j]`` radians.

    freq: 32 frequencies (radians per position).  axis: the axis of each pair (time, height,
    width, ...; all 0 for text).  pairing: "adjacent", pairs (2j, 2j + 1), or "halves", pairs
    (j, j + 32).
    """

    def __init__(self, freq, axis=None, pairing: str = "adjacent"):
        freq = [float(f) for f in freq]
        axis = [int(a) for a in axis] if axis is not None else [0] * ROPE_PAIRS
        if not (len(freq) == ROPE_PAIRS and len(axis) == ROPE_PAIRS):
            raise ValueError(f"a rotary has {ROPE_PAIRS} frequencies and axes")
        if not all(0 <= a < ula.MAX_AXES for a in axis):
            raise ValueError(f"an axis is in [0, {ula.MAX_AXES})")
        if pairing not in _PAIRINGS:
            raise ValueError(f"pairing is one of {sorted(_PAIRINGS)}")
        self.n_axes = max(axis) + 1
        self.config = ula.ula_rotary()
        self.config.n_axes, self.config.pairing = self.n_axes, _PAIRINGS[pairing]
        self.config.freq[:] = freq
        self.config.axis[:] = axis


def _positions(pos: torch.Tensor, rotary: Rotary, n: int):
    if pos.dtype != torch.int32:
        raise ValueError("positions are int32")
    if pos.dim() == 1:
        pos = pos[None]
    if not (pos.dim() == 2 and pos.shape[0] >= rotary.n_axes and pos.shape[1] == n):
        raise ValueError("positions are [axes][tokens]")
    if pos.stride(1) != 1 and n > 1:
        pos = pos.contiguous()
    return pos


@_on_stream
def rotate(x: torch.Tensor, pos: torch.Tensor, rotary: Rotary, *, out: torch.Tensor | None = None,
           inverse: bool = False) -> torch.Tensor:
    """Turns the rope channels of x [tokens][heads][64] (or [tokens][64]); bf16, f16 or f32.

    pos: int32 [axes][tokens] (or [tokens]).  out: x itself (in place) or another tensor of x's
    shape and type, such as the last 64 channels of the queries that ``attend`` reads.
    inverse turns back; it is also the gradient.
    """
    if not (x.dim() in (2, 3) and x.shape[-1] == ROW_ROPE and x.dtype in _TYPES):
        raise ValueError(f"x is [tokens][heads][{ROW_ROPE}] of bf16, f16 or f32")
    n, heads = x.shape[0], x.shape[1] if x.dim() == 3 else 1
    pos = _positions(pos, rotary, n)
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    if not (out.shape == x.shape and out.dtype == x.dtype and out.stride(-1) == 1):
        raise ValueError("out has x's shape and type, and dense channels")
    if x.stride(-1) != 1:
        x = x.contiguous()
    handle = _stream_of(x, pos, out)
    three = x.dim() == 3
    ula.ula_rows_rotate(rotary.config, ula.ROTATE_INVERSE if inverse else 0, pos.data_ptr(),
                        pos.stride(0), n, heads, _TYPES[x.dtype],
                        x.data_ptr(), x.stride(0), x.stride(1) if three else 0,
                        out.data_ptr(), out.stride(0), out.stride(1) if three else 0, handle)
    return out


@_on_stream
def pack(latent: torch.Tensor, rope: torch.Tensor, pos: torch.Tensor, rotary: Rotary,
         rows: torch.Tensor | None = None) -> torch.Tensor:
    """Packs tokens into cache rows: latent [n][512] (bf16, f16 or f32) to e4m3 with a scale per
    128 channels, rope [n][64] (the latent's type) turned at its positions and stored in bf16.

    rows: uint8 [n][656] to write (rows may lie apart, such as one layer [:, j] of the
    [n][L][656] that ``UlaCache.alloc`` takes), or None for a new tensor.  Returns rows.
    """
    n = latent.shape[0]
    if not (latent.dtype in _TYPES and latent.shape == (n, ROW_LATENT)):
        raise ValueError(f"latent is [tokens][{ROW_LATENT}] of bf16, f16 or f32")
    if not (rope.dtype == latent.dtype and rope.shape == (n, ROW_ROPE)):
        raise ValueError(f"rope is [tokens][{ROW_ROPE}] of the latent's type")
    if latent.stride(1) != 1:
        latent = latent.contiguous()
    if rope.stride(1) != 1:
        rope = rope.contiguous()
    pos = _positions(pos, rotary, n)
    if rows is None:
        rows = torch.empty((n, ROW_BYTES), dtype=torch.uint8, device=latent.device)
    if not (rows.dtype == torch.uint8 and rows.shape == (n, ROW_BYTES)
          and rows.stride(1) == 1 and (n < 2 or rows.stride(0) >= ROW_BYTES)):
        raise ValueError(f"rows is uint8 [tokens][{ROW_BYTES}]")
    handle = _stream_of(latent, rope, pos, rows)
    ula.ula_rows_pack(rotary.config, pos.data_ptr(), pos.stride(0), n, _TYPES[latent.dtype],
                      latent.data_ptr(), latent.stride(0), rope.data_ptr(), rope.stride(0),
                      rows.data_ptr(), rows.stride(0) if n > 1 else ROW_BYTES, handle)
    return rows


@_on_stream
def attend(q: torch.Tensor, rows: torch.Tensor, entry_row: torch.Tensor, softmax_scale: float, *,
           own_rows: torch.Tensor | None = None, out: torch.Tensor | None = None,
           lse: torch.Tensor | None = None):
    """Attention of query tokens over the rows a step gathered; returns (out, lse).

    q: bf16 [R][Q][H][576] (512 latent channels, then 64 rope channels, already turned).
    rows: uint8 [cap][656], one layer of ``step_group``'s output.  entry_row: int32 [R][Q][K],
    ``step_group``'s entry rows; entries outside [0, cap), such as the -1 of a pad, select
    nothing.  own_rows: uint8 [R][Q][656], the step's own tokens: query token i of a request
    also sees own rows 0..i.
    out: bf16 [R][Q][H][512], lse: float32 [R][Q][H], ln of the sum of exp(logits); a query token
    that selects nothing gets 0 and -inf.
    """
    if not (q.dim() == 4 and q.shape[3] == ROW_LATENT + ROW_ROPE and q.dtype == torch.bfloat16):
        raise ValueError(f"q is bf16 [requests][query tokens][heads][{ROW_LATENT + ROW_ROPE}]")
    R, Q, H, _ = q.shape
    if not (rows.dtype == torch.uint8 and rows.dim() == 2 and rows.shape[1] == ROW_BYTES
          and rows.is_contiguous()):
        raise ValueError(f"rows is contiguous uint8 [rows][{ROW_BYTES}]")
    if not (entry_row.dtype == torch.int32 and entry_row.dim() == 3
          and entry_row.shape[:2] == (R, Q)):
        raise ValueError("entry_row is int32 [requests][query tokens][k]")
    if not entry_row.is_contiguous():
        entry_row = entry_row.contiguous()
    sq = q.stride()
    if sq[3] != 1 or sq[0] % 8 or sq[1] % 8 or sq[2] % 8 or q.data_ptr() % 16:
        q = q.clone(memory_format=torch.contiguous_format)
        sq = q.stride()
    K = entry_row.shape[2]
    own, so = None, (0, 0)
    if own_rows is not None:
        if not (own_rows.dtype == torch.uint8 and own_rows.shape == (R, Q, ROW_BYTES)
              and own_rows.stride(2) == 1):
            raise ValueError(f"own_rows is uint8 [requests][query tokens][{ROW_BYTES}]")
        own, so = own_rows.data_ptr(), own_rows.stride()
    if out is None:
        out = torch.empty((R, Q, H, ROW_LATENT), dtype=torch.bfloat16, device=q.device)
    else:
        if not (out.dtype == torch.bfloat16 and out.shape == (R, Q, H, ROW_LATENT)
              and out.is_contiguous()):
            raise ValueError(f"out is contiguous bf16 [{R}][{Q}][{H}][{ROW_LATENT}]")
    if lse is None:
        lse = torch.empty((R, Q, H), dtype=torch.float32, device=q.device)
    else:
        if not (lse.dtype == torch.float32 and lse.shape == (R, Q, H) and lse.is_contiguous()):
            raise ValueError(f"lse is contiguous float32 [{R}][{Q}][{H}]")
    handle = _stream_of(q, rows, entry_row, out, lse, *(() if own_rows is None else (own_rows,)))
    nbytes = ula.ula_rows_attend_workspace(R, Q, H, K, own is not None)
    space = torch.empty(nbytes, dtype=torch.uint8, device=q.device) if nbytes else None
    ula.ula_rows_attend(ula.ula_attend_args(
        q.data_ptr(), sq[0], sq[1], sq[2], rows.data_ptr(), entry_row.data_ptr(), own, so[0],
        so[1], out.data_ptr(), lse.data_ptr(), space.data_ptr() if nbytes else None, nbytes,
        rows.shape[0], R, Q, H, K, softmax_scale), handle)
    return out, lse


@_on_stream
def join(outs, lses, *, out: torch.Tensor | None = None, lse: torch.Tensor | None = None):
    """Joins partial results over disjoint rows (at most 8 parts): lists of ``attend``'s outs
    (bf16 [...][512]) and lses (float32 [...]).  Returns (out, lse); a part with lse -inf counts
    for nothing.  out and lse may be one of the parts."""
    if not (1 <= len(outs) <= ula.MAX_PARTS and len(outs) == len(lses)):
        raise ValueError(f"1 to {ula.MAX_PARTS} parts, an out and an lse of each")
    shape = outs[0].shape
    if not (len(shape) >= 1 and shape[-1] == ROW_LATENT):
        raise ValueError(f"a part's out is [...][{ROW_LATENT}]")
    for o, z in zip(outs, lses):
        if not (o.dtype == torch.bfloat16 and o.shape == shape and o.is_contiguous()):
            raise ValueError(f"a part's out is contiguous bf16 [...][{ROW_LATENT}], all of one shape")
        if not (z.dtype == torch.float32 and z.shape == shape[:-1] and z.is_contiguous()):
            raise ValueError("a part's lse is contiguous float32 of its out's shape without the channels")
    device = outs[0].device
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=device)
    else:
        if not (out.dtype == torch.bfloat16 and out.shape == shape and out.is_contiguous()):
            raise ValueError("out is contiguous bf16 of the parts' shape")
    if lse is None:
        lse = torch.empty(shape[:-1], dtype=torch.float32, device=device)
    else:
        if not (lse.dtype == torch.float32 and lse.shape == shape[:-1] and lse.is_contiguous()):
            raise ValueError("lse is contiguous float32 of the parts' shape")
    handle = _stream_of(*outs, *lses, out, lse)
    ula.ula_rows_join([o.data_ptr() for o in outs], [z.data_ptr() for z in lses],
                      lses[0].numel(), out.data_ptr(), lse.data_ptr(), handle)
    return out, lse


def sync(stream: torch.cuda.Stream | None = None) -> None:
    """Waits for the stream; raises the first error these operators latched on the device."""
    s = stream if stream is not None else torch.cuda.current_stream()
    ula.ula_rows_sync(s.cuda_stream)
