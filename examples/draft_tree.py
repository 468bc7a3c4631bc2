"""Decoding with trees of drafted tokens over a residency cache with a budget, on one GPU.

A few requests with histories in a ``UlaCache`` decode for a few steps.  Per step every request has a
tree of drafted tokens: node 0 is the token accepted last, every other node hangs on an earlier one.
Per step and layer the nodes' keys are normed and packed into rows, the queries' heads are normed and
turned (both at the position of the node's depth), the cache makes the selected rows resident and
gathers them, the nodes attend over them and over their branches, and the attention's weights are
accumulated by address.  Then a branch is accepted (at random here, where a model would compare its
samples with the drafts) and its rows are appended; a request with more tokens than its budget gives up
those whose weights are smallest.

    python examples/draft_tree.py [--check]

--check compares every layer's output, the accumulated weights and what was given up with a computation in 64 bits.
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

REQ, CTX, NODES, K, HEADS = 3, 2000, 7, 128, 20
GROUPS, LAYERS, WINDOW, FIRST, BUDGET = 2, 2, 16, 4, 1900
SCALE, EPS = (128 + 64) ** -0.5, 1e-6


def unpack64(r: torch.Tensor):
    """Rows [n][656] as latents and rope channels in float64."""
    latent = r[:, :512].contiguous().view(torch.float8_e4m3fn).double().view(-1, 4, 128)
    scale = r[:, 512:528].contiguous().view(torch.float32).double()
    return ((latent * scale[..., None]).flatten(1),
            r[:, 528:].contiguous().view(torch.bfloat16).double())


class Model:
    """Stand-ins for what a model's projections would produce, from a seed, and its norms' weights."""

    def __init__(self, seed: int):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.rotary = rows.Rotary(10000.0 ** (-np.arange(32) / 32), pairing="halves")
        self.q_weight = 1 + 0.1 * self.randn(576)
        self.k_weight, self.rope_weight = 1 + 0.1 * self.randn(512), 1 + 0.1 * self.randn(64)

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(torch.bfloat16)

    def pack_tokens(self, time: torch.Tensor, out: torch.Tensor) -> torch.Tensor:
        """Packs tokens for every layer of out [n][L][656]."""
        pos = time.to(torch.int32)
        for j in range(out.shape[1]):
            rows.pack_norm(3 * self.randn(len(time), 512), self.randn(len(time), 64), self.k_weight, pos, self.rotary,
                           out[:, j], rope_weight=self.rope_weight, eps=EPS)
        return out

    def queries(self, time: torch.Tensor) -> torch.Tensor:
        """[REQ][NODES][HEADS][576], every head normed, its rope channels turned, in place."""
        q = 2 * self.randn(REQ * NODES, HEADS, 576)
        rows.norm_rotate(q, self.q_weight, time.to(torch.int32), self.rotary, eps=EPS, out=q)
        return q.view(REQ, NODES, HEADS, 576)


def path_of(parent, node: int) -> list[int]:
    """The node and its ancestors, the root first."""
    path = [node]
    while parent[path[-1]] >= 0:
        path.append(int(parent[path[-1]]))
    return path[::-1]


def run(steps: int = 4, seed: int = 0, check: bool = False) -> tuple[float, float]:
    """Decodes; returns the largest error of an output channel against 64 bits, and that of an address's accumulated weights as
    a part of them (with check)."""
    model = Model(seed)
    rng = np.random.default_rng(seed)
    total = REQ * (CTX + steps * NODES)
    cache = UlaCache(row_bytes=656, layers_per_group=[LAYERS] * GROUPS, gpu_slots=total // 2, host_slots=total,
                     ring_buckets=4, max_logical=total, max_entries=REQ * NODES * K)
    try:
        owned = [[] for _ in range(REQ)]     # each request's logical addresses, oldest first
        length = [0] * REQ                   # its tokens so far, those given up among them
        store = [[] for _ in range(GROUPS)]  # (check) every row ever appended, by address
        scores = torch.zeros(total, device="cuda")
        want_scores = torch.zeros(total, dtype=torch.float64, device="cuda")

        def append(r: int, group_rows):
            n = len(group_rows[0])
            base = cache.alloc(n, torch.cat([g.reshape(-1) for g in group_rows]))
            cache.sync()  # the rows' tensor is this function's own
            owned[r].extend(range(base, base + n))
            length[r] += n
            for g in range(GROUPS):
                store[g].append(group_rows[g].clone())

        for r in range(REQ):
            append(r, [model.pack_tokens(torch.arange(CTX, device="cuda"),
                                         torch.empty(CTX, LAYERS, 656, dtype=torch.uint8, device="cuda"))
                       for _ in range(GROUPS)])
        entry_row = torch.empty(REQ * NODES * K, dtype=torch.int32, device="cuda")
        req_off = torch.empty(REQ + 1, dtype=torch.int32, device="cuda")
        worst = 0.0
        for _ in range(steps):
            parents = np.stack([[-1] + [int(rng.integers(0, i)) for i in range(1, NODES)] for _ in range(REQ)])
            parent = torch.from_numpy(parents.astype(np.int32)).cuda()
            time = torch.tensor([length[r] + len(path_of(parents[r], i)) - 1 for r in range(REQ) for i in range(NODES)],
                                device="cuda")
            new_rows = []
            for g in range(GROUPS):
                # each node selects the recent window and K - WINDOW others of the request's tokens
                sel = np.stack([[np.concatenate([owned[r][-WINDOW:], rng.choice(owned[r][:-WINDOW], K - WINDOW, replace=False)])
                                 for _ in range(NODES)] for r in range(REQ)]).astype(np.int32)
                sel_d = torch.from_numpy(sel).cuda()
                out = cache.out_buffer(g, REQ * NODES * K)
                cache.step_group(g, sel_d, out, entry_row, req_off)
                entry = entry_row.view(REQ, NODES, K)
                own = model.pack_tokens(time, torch.empty(REQ * NODES, LAYERS, 656, dtype=torch.uint8, device="cuda"))
                for j in range(LAYERS):
                    q = model.queries(time)
                    own_j = own[:, j].unflatten(0, (REQ, NODES))
                    o, lse = rows.attend_tree(q, out[j], entry, SCALE, own_j, parent)
                    rows.score(scores, q, out[j], entry, sel_d, lse, SCALE)
                    if check:
                        every = torch.cat(store[g])[:, j]
                        for r in range(REQ):
                            for i in range(NODES):
                                picked = every[sel_d[r, i].long()]
                                latent, rope = unpack64(torch.cat([picked, own_j[r, path_of(parents[r], i)]]))
                                p = torch.softmax((q[r, i].double() @ torch.cat([latent, rope], 1).t()) * SCALE, dim=1)
                                worst = max(worst, float((o[r, i].double() - p @ latent).abs().max()))
                                want_scores.index_add_(0, sel_d[r, i].long(), p[:, :K].sum(0))
                new_rows.append(own.view(REQ, NODES, LAYERS, 656))
            for r in range(REQ):  # the accepted branch joins the cache
                branch = path_of(parents[r], int(rng.integers(0, NODES)))
                append(r, [new_rows[g][r, branch] for g in range(GROUPS)])
            # what is over the budget leaves
            longest = max(len(o) for o in owned)
            address = torch.tensor([o + [-1] * (longest - len(o)) for o in owned], dtype=torch.int32).cuda()
            count = torch.tensor([len(o) for o in owned], dtype=torch.int32).cuda()
            kept, dropped = rows.evict(scores, address, count, BUDGET, first=FIRST, last=WINDOW)
            if check:
                for r in range(REQ):
                    gone = dropped[r][dropped[r] >= 0].long()
                    middle = torch.tensor(owned[r][FIRST:len(owned[r]) - WINDOW], device="cuda")
                    stay = middle[~torch.isin(middle, gone)]
                    assert torch.isin(gone, middle).all() and len(gone) == max(0, len(owned[r]) - BUDGET)
                    assert len(gone) == 0 or scores[gone].max() <= scores[stay].min()
            cache.free_each(dropped)
            owned = [row[row >= 0].tolist() for row in kept.cpu()]
        cache.sync()
        rows.sync()
        # (an address that no node selected has 0, and anything else there counts as infinitely wrong)
        off = torch.where(scores == want_scores, 0.0, (scores.double() - want_scores).abs() / want_scores)
        return worst, float(off.max()) if check else 0.0
    finally:
        cache.close()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--check", action="store_true")
    ap.add_argument("--steps", type=int, default=4)
    a = ap.parse_args()
    err, off = run(a.steps, check=a.check)
    print(f"{a.steps} steps of {REQ} requests x {NODES} drafted tokens, {GROUPS} x {LAYERS} layers, {BUDGET} tokens kept"
          + (f"; largest error against 64 bits {err:.2e}, of an address's weights {off:.2e} of them" if a.check else ""))
