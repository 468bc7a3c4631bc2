"""Operators on the cache's FP8 rows: rotary positions, packing, attention, joining, eviction.

A row is 656 bytes: 512 e4m3 codes (the latent), 4 fp32 scales (one for each block of
128 channels), 64 bf16 rope channels.  A decode layer packs its new tokens into rows
(``pack``, whose rows go to ``UlaCache.alloc``), turns its queries' rope channels
(``rotate``), attends over the rows that ``UlaCache.step_group`` gathered (``attend``) and
joins partial results over disjoint rows (``join``: ``UlaTP``'s local and remote rows).  Where
queries and keys are normed first, ``norm_rotate`` and ``pack_norm`` do that in the same pass; where
a step verifies a tree of drafted tokens, ``attend_tree`` is its attention; and where a request has a
budget, ``score`` accumulates the attention's weights by logical address and ``evict`` picks those that
leave (for ``UlaCache.free_each``).

Every step runs in the CUDA library through the C ABI; ``_build/_rows.so`` checks and marshals
the arguments (in C++: a decode step makes four of these calls per layer).  Calls run on
``stream`` (default: the current stream of the tensors' device) and return without waiting.
Wrong shapes, types or devices raise ValueError, errors of the C ABI ``ula.UlaError``.  Nothing
is recorded for autograd: tensors that require a gradient are refused outside ``torch.no_grad()``, and so are
dual tensors of forward-mode differentiation.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os

import torch

from . import ula
from .ula import ROPE_PAIRS


def _load():
    path = os.path.join(os.path.dirname(ula.LIB_PATH), "_rows.so")
    if not os.path.exists(path):
        raise ImportError(f"binding not built: {path} (run __graft_entry__.build())")
    loader = importlib.machinery.ExtensionFileLoader("_rows", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_rows", path, loader=loader))
    loader.exec_module(module)
    return module


_rows = _load()
_PAIRINGS = {"adjacent": ula.PAIR_ADJACENT, "halves": ula.PAIR_HALVES}


def _on(stream: torch.cuda.Stream, call, *args):
    """Runs a call (copies and outputs it makes included) on another stream than the current
    one.  The tensors handed in, which another stream's allocator may own, are recorded there,
    so that their memory is not handed out again while the call still runs."""
    with torch.cuda.stream(stream):
        result = call(*args)
    for t in _tensors(args):
        t.record_stream(stream)
    return result


def _tensors(v):
    if isinstance(v, torch.Tensor):
        yield v
    elif isinstance(v, (list, tuple)):
        for x in v:
            yield from _tensors(x)


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
        if len(freq) != ROPE_PAIRS or len(axis) != ROPE_PAIRS:
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


def rotate(x: torch.Tensor, pos: torch.Tensor, rotary: Rotary, *, out: torch.Tensor | None = None,
           inverse: bool = False, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Turns the rope channels of x [tokens][heads][64] (or [tokens][64]); bf16, f16 or f32.

    pos: int32 [axes][tokens] (or [tokens]).  out: x itself (in place) or another tensor of x's
    shape and type, such as the last 64 channels of the queries that ``attend`` reads; its tokens
    and heads may not share memory.
    inverse turns back; it is also the gradient (for a backward function of the caller's).
    """
    if stream is not None:
        return _on(stream, _rows.rotate, x, pos, rotary.config, out, bool(inverse))
    return _rows.rotate(x, pos, rotary.config, out, bool(inverse))


def pack(latent: torch.Tensor, rope: torch.Tensor, pos: torch.Tensor, rotary: Rotary,
         rows: torch.Tensor | None = None, *,
         stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Packs tokens into cache rows: latent [n][512] (bf16, f16 or f32) to e4m3 with a scale per
    128 channels, rope [n][64] (the latent's type) turned at its positions and stored in bf16.

    rows: uint8 [n][656] to write (rows may lie apart, such as one layer [:, j] of the
    [n][L][656] that ``UlaCache.alloc`` takes), or None for a new tensor.  Returns rows.
    """
    if stream is not None:
        return _on(stream, _rows.pack, latent, rope, pos, rotary.config, rows)
    return _rows.pack(latent, rope, pos, rotary.config, rows)


def norm_rotate(x: torch.Tensor, weight: torch.Tensor, pos: torch.Tensor, rotary: Rotary, *,
                eps: float = 1e-6, at: int | None = None, out: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Norms the heads of x [tokens][heads][width] (or [tokens][width]; bf16, f16 or f32; width 64 to
    1024) and turns their rope channels, in one pass: y = x / sqrt(mean(x^2) + eps) * weight over
    a head's channels, then y's channels at..at + 63 (default: the last 64) as by ``rotate``.  In float32,
    sums of squares too: channels up to 5e17 (from 1e-15, a head's largest, where eps is below 1e-30).

    weight: [width] of x's type or float32.  pos: int32 [axes][tokens] (or [tokens]).  out: x itself
    (in place) or another tensor of x's shape and type, whose tokens and heads may not share memory.
    """
    if stream is not None:
        return _on(stream, _rows.norm_rotate, x, weight, pos, rotary.config, eps, at, out)
    return _rows.norm_rotate(x, weight, pos, rotary.config, eps, at, out)


def pack_norm(latent: torch.Tensor, rope: torch.Tensor, latent_weight: torch.Tensor, pos: torch.Tensor,
              rotary: Rotary, rows: torch.Tensor | None = None, *,
              rope_weight: torch.Tensor | None = None, eps: float = 1e-6,
              stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """``pack`` with the key's norm in the same pass: the latents become x / sqrt(mean(x^2) + eps) *
    latent_weight before they are quantised, and with rope_weight the rope channels as much before they
    are turned.  Weights: [512] and [64], of the latent's type or float32.  Channels may be as large as ``norm_rotate``'s."""
    if stream is not None:
        return _on(stream, _rows.pack_norm, latent, rope, latent_weight, pos, rotary.config, eps, rope_weight, rows)
    return _rows.pack_norm(latent, rope, latent_weight, pos, rotary.config, eps, rope_weight, rows)


def attend(q: torch.Tensor, rows: torch.Tensor, entry_row: torch.Tensor, softmax_scale: float, *,
           own_rows: torch.Tensor | None = None, out: torch.Tensor | None = None,
           lse: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """Attention of query tokens over the rows a step gathered; returns (out, lse).

    q: bf16 [R][Q][H][576] (512 latent channels, then 64 rope channels, already turned).
    rows: uint8 [cap][656], one layer of ``step_group``'s output.  entry_row: int32 [R][Q][K],
    ``step_group``'s entry rows; entries outside [0, cap), such as the -1 of a pad, select
    nothing.  own_rows: uint8 [R][Q][656], the step's own tokens: query token i of a request
    also sees own rows 0..i.
    out: bf16 [R][Q][H][512], lse: float32 [R][Q][H], ln of the sum of exp(logits); a query token
    that selects nothing gets 0 and -inf.
    """
    if stream is not None:
        return _on(stream, _rows.attend, q, rows, entry_row, softmax_scale, own_rows, out, lse)
    return _rows.attend(q, rows, entry_row, softmax_scale, own_rows, out, lse)


def attend_tree(q: torch.Tensor, rows: torch.Tensor, entry_row: torch.Tensor, softmax_scale: float,
                own_rows: torch.Tensor, parent: torch.Tensor, *, out: torch.Tensor | None = None,
                lse: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """Attention of a tree of drafted tokens over the rows a step gathered; returns (out, lse).

    As ``attend``, with query token i of a request as node i of its tree (at most 64 nodes): it sees
    its entries' rows and the own rows of i, parent[r, i], that node's parent, and so on.
    parent: int32 [R][Q]; a value that is not an earlier node's, such as -1, stands for none.
    entry_row: int32 [R][Q][K], a list for each node, or [R][K], one that all nodes of a request's
    tree share (its rows are then read once for all their query heads).
    An own row with NaN codes or scales that are not finite gives NaN to the nodes that see it, and
    counts for nothing for the others.
    """
    if stream is not None:
        return _on(stream, _rows.attend_tree, q, rows, entry_row, softmax_scale, own_rows, parent, out, lse)
    return _rows.attend_tree(q, rows, entry_row, softmax_scale, own_rows, parent, out, lse)


def join(outs, lses, *, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
         stream: torch.cuda.Stream | None = None):
    """Joins partial results over disjoint rows (at most 8 parts): lists of ``attend``'s outs
    (bf16 [...][512]) and lses (float32 [...]).  Returns (out, lse); a part with lse -inf counts
    for nothing.  out and lse may be one of the parts."""
    if stream is not None:
        return _on(stream, _rows.join, outs, lses, out, lse)
    return _rows.join(outs, lses, out, lse)


def score(scores: torch.Tensor, q: torch.Tensor, rows: torch.Tensor, entry_row: torch.Tensor,
          address: torch.Tensor, lse: torch.Tensor, softmax_scale: float, *,
          stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Accumulates attention weights by logical address, in place: for every query token's entry e,
    scores[address[e]] += sum over heads of exp(logit[e] - lse).  Returns scores.

    scores: float32 [addresses].  q, rows, entry_row: ``attend``'s (or ``attend_tree``'s, [R][K] too).
    address: int32 of entry_row's shape, the selection that ``step_group`` got.  lse: float32
    [R][Q][H], the attention's (joined with other parts: weights of the whole).  Entries whose row or
    address is out of range count for nothing, and so do query tokens whose lse is -inf.  The result does
    not depend on the order in which an address's weights are added: they are summed as whole numbers of
    2^(-2e), with 2^(62 - e) the power of two at or above R * Q * H * K (4 at least), and added to the score once.
    """
    if stream is not None:
        return _on(stream, _rows.score, scores, q, rows, entry_row, address, lse, softmax_scale)
    return _rows.score(scores, q, rows, entry_row, address, lse, softmax_scale)


def evict(scores: torch.Tensor, address: torch.Tensor, length: torch.Tensor, budget: int, *,
          first: int = 0, last: int = 0, kept: torch.Tensor | None = None,
          dropped: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None):
    """Which of each request's logical addresses stay within a budget; returns (kept, dropped).

    address: int32 [R][N], a request's addresses, oldest first, of which length [R] (int32) count.
    The first ``first`` and the last ``last`` stay, and of the others those with the largest
    scores (float32 [addresses]), min(length, budget) in all; where scores are equal the older ones
    leave.  kept: int32 [R][budget], dropped: int32 [R][max(N - budget, 0)] (for
    ``UlaCache.free_each``), in the list's order, -1 behind; neither may share memory with an input or the other.
    """
    if stream is not None:
        return _on(stream, _rows.evict, scores, address, length, budget, first, last, kept, dropped)
    return _rows.evict(scores, address, length, budget, first, last, kept, dropped)


def sync(stream: torch.cuda.Stream | None = None) -> None:
    """Waits for the stream (default: the current one).  Raises ``ula.UlaError`` if a bounded wait of
    an ``attend``, ``attend_tree`` or ``score`` on the stream's device, on this stream or another, has run out since this
    stream's last sync; the call's outputs are then not valid."""
    s = stream if stream is not None else torch.cuda.current_stream()
    with torch.cuda.device(s.device):
        ula.ula_rows_sync(s.cuda_stream)
