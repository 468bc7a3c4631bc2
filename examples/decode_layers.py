"""Sparse-attention decode steps over a residency cache, end to end on one GPU.

A few requests with histories in a ``UlaCache`` (some of each history in HBM, the rest in pinned
host memory) decode for a few steps.  Per step and layer: the new tokens' latents and rope
channels are packed into rows (time, height and width positions), the queries' rope channels are
turned, the cache makes the selected rows resident and gathers them, and the queries attend over
them and over the step's own rows; a prefix that all requests share is kept outside the cache,
attended to separately and joined in.  After the step the accepted tokens' rows are appended.

    python examples/decode_layers.py [--check]

--check compares every layer's output with a dense computation in 64 bits.
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from serving_step_sparse_gb300 import rows  # noqa: E402
from serving_step_sparse_gb300.cache import UlaCache  # noqa: E402

REQ, CTX, PREFIX, Q, K, HEADS = 4, 1500, 96, 3, 256, 20
GROUPS, LAYERS, WINDOW = 2, 3, 32
SCALE = (128 + 64) ** -0.5


def make_rotary() -> rows.Rotary:
    """Base 10,000; time, height and width turn consecutive sections of the 32 pairs."""
    freq = 10000.0 ** (-np.arange(32) / 32)
    return rows.Rotary(freq, [0] * 12 + [1] * 10 + [2] * 10, "halves")


def unpack64(r: torch.Tensor):
    """Rows [n][656] as latents and rope channels in float64."""
    latent = r[:, :512].contiguous().view(torch.float8_e4m3fn).double().view(-1, 4, 128)
    scale = r[:, 512:528].contiguous().view(torch.float32).double()
    return ((latent * scale[..., None]).flatten(1),
            r[:, 528:].contiguous().view(torch.bfloat16).double())


class Model:
    """Stand-ins for what a model's projections would produce, from a seed."""

    def __init__(self, seed: int):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.rotary = make_rotary()

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(torch.bfloat16)

    def positions(self, time: torch.Tensor) -> torch.Tensor:
        """[3][n]: text moves in time only, every 7th token is part of a 16 x 16 frame."""
        frame = time % 7 == 0
        return torch.stack([time, torch.where(frame, time // 16 % 16, time),
                            torch.where(frame, time % 16, time)]).to(torch.int32)

    def pack_tokens(self, time: torch.Tensor, out: torch.Tensor) -> torch.Tensor:
        """Packs tokens for every layer of out [n][L][656]."""
        pos = self.positions(time)
        for j in range(out.shape[1]):
            rows.pack(self.randn(len(time), 512), self.randn(len(time), 64), pos, self.rotary,
                      out[:, j])
        return out

    def queries(self, time: torch.Tensor) -> torch.Tensor:
        """[REQ][Q][HEADS][576], the rope channels turned in place."""
        q = self.randn(REQ * Q, HEADS, 576)
        rope = q[..., 512:]
        rows.rotate(rope, self.positions(time), self.rotary, out=rope)
        return q.view(REQ, Q, HEADS, 576)


def dense64(q, history, own, prefix):
    """One request's attention over rows [n][656], own rows 0..i and the prefix, in 64 bits."""
    out = []
    for i in range(Q):
        latent, rope = unpack64(torch.cat([history[i], own[:i + 1], prefix]))
        z = (q[i].double() @ torch.cat([latent, rope], 1).t()) * SCALE
        out.append(torch.softmax(z, dim=1) @ latent)
    return torch.stack(out)


def run(steps: int = 3, seed: int = 0, check: bool = False) -> float:
    """Decodes; returns the largest error of an output channel against 64 bits (with check)."""
    model = Model(seed)
    rng = np.random.default_rng(seed)
    total = REQ * (CTX + steps * Q)
    cache = UlaCache(row_bytes=656, layers_per_group=[LAYERS] * GROUPS, gpu_slots=total // 2,
                     host_slots=total, ring_buckets=4, max_logical=total, max_entries=REQ * Q * K)
    try:
        # prompts: packed layer by layer, then handed to the cache group by group
        owned = [[] for _ in range(REQ)]     # each request's logical addresses, oldest first
        store = [[] for _ in range(GROUPS)]  # (check) every row ever appended, by address
        # (the prefix layer by layer: attend takes one layer's rows one after the other)
        prefix = [model.pack_tokens(torch.arange(PREFIX, device="cuda"),
                                    torch.empty(LAYERS, PREFIX, 656, dtype=torch.uint8,
                                                device="cuda").transpose(0, 1))
                  for _ in range(GROUPS)]

        def append(r: int, group_rows):
            n = len(group_rows[0])
            base = cache.alloc(n, torch.cat([g.reshape(-1) for g in group_rows]))
            cache.sync()  # the rows' tensor is this function's own
            owned[r].extend(range(base, base + n))
            for g in range(GROUPS):
                store[g].append(group_rows[g].clone())

        for r in range(REQ):
            time = torch.arange(PREFIX, PREFIX + CTX, device="cuda")
            append(r, [model.pack_tokens(time, torch.empty(CTX, LAYERS, 656, dtype=torch.uint8,
                                                           device="cuda")) for _ in range(GROUPS)])
        prefix_entries = torch.arange(PREFIX, dtype=torch.int32, device="cuda").expand(
            REQ, Q, PREFIX).contiguous()
        entry_row = torch.empty(REQ * Q * K, dtype=torch.int32, device="cuda")
        req_off = torch.empty(REQ + 1, dtype=torch.int32, device="cuda")
        worst = 0.0
        for _ in range(steps):
            time = torch.cat([PREFIX + len(owned[r]) + torch.arange(Q, device="cuda")
                              for r in range(REQ)])
            accepted = rng.integers(1, Q + 1, REQ)
            new_rows = []
            for g in range(GROUPS):
                # each query token selects its recent window and K - WINDOW others of its history
                sel = np.stack([[np.concatenate([owned[r][-WINDOW:], rng.choice(
                    owned[r][:-WINDOW], K - WINDOW, replace=False)]) for _ in range(Q)]
                    for r in range(REQ)]).astype(np.int32)
                out = cache.out_buffer(g, REQ * Q * K)
                cache.step_group(g, torch.from_numpy(sel).cuda(), out, entry_row, req_off)
                own = model.pack_tokens(time, torch.empty(REQ * Q, LAYERS, 656, dtype=torch.uint8,
                                                          device="cuda"))
                for j in range(LAYERS):
                    q = model.queries(time)
                    own_j = own[:, j].unflatten(0, (REQ, Q))
                    part = rows.attend(q, out[j], entry_row.view(REQ, Q, K), SCALE, own_rows=own_j)
                    shared = rows.attend(q, prefix[g][:, j], prefix_entries, SCALE)
                    o, _ = rows.join([part[0], shared[0]], [part[1], shared[1]])
                    if check:
                        every = torch.cat(store[g])[:, j]
                        for r in range(REQ):
                            picked = [every[torch.from_numpy(sel[r, i].astype(np.int64)).cuda()]
                                      for i in range(Q)]
                            want = dense64(q[r], picked, own_j[r], prefix[g][:, j])
                            worst = max(worst, float((o[r].double() - want).abs().max()))
                new_rows.append(own.view(REQ, Q, LAYERS, 656))
            for r in range(REQ):  # the accepted tokens join the cache
                append(r, [new_rows[g][r, :accepted[r]] for g in range(GROUPS)])
        cache.sync()
        rows.sync()
        return worst
    finally:
        cache.close()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--check", action="store_true")
    ap.add_argument("--steps", type=int, default=3)
    a = ap.parse_args()
    err = run(a.steps, check=a.check)
    print(f"{a.steps} steps of {REQ} requests x {Q} tokens, {GROUPS} x {LAYERS} layers"
          + (f"; largest error against 64 bits {err:.2e}" if a.check else ""))
