"""The operators around a drafted step (normed positions and packing, attention of a tree, accumulated
weights, eviction) against plain implementations in 64 bits.

Tolerances, derived from the number formats (those of the attention: test_gpu_rows.py):
  * a norm's sum of squares has at most 131 fp32 roundings in a row (width 1,024: 128 products of a lane
    and 3 steps), half of which reach the root: 2^-24 * 66; division, sum, root and two products add
    5 * 2^-24: every normed value is off by at most 2^-17 of its size before it is rounded;
  * an attention weight is off by a factor of e^d, with d the logit's error (2^-20 * sum |q k| * scale), the
    rounding of lse * log2(e) and of the difference (2^-22 * (|z| + |lse|) in all) and 2^-22 from the
    exponential; sums of heads in fp32 lose 2^-16 at most (130 heads in a row: 130 * 2^-24), the
    fixed point half of its unit, 2^-(64 - bits), a weight, and the score is rounded twice (2^-23).
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from tests.test_gpu_rows import (DT, E4M3, HALF_ULP, SCALE, SMALLEST, attend64, attend_case, check_attend,
                                 make_rotary, positions, random_rows, turned, unpack)

pytestmark = pytest.mark.gpu

NORM = 2.0 ** -17


# ------------------------------------------------------------------------------- a tree

def branches(parent):
    """For each node its own place and its ancestors'."""
    out = []
    for i in range(len(parent)):
        path, a = [i], i
        while 0 <= parent[a] < a:
            a = int(parent[a])
            path.append(a)
        out.append(sorted(path))
    return out


def tree64(q, rows, entry, scale, own, parent):
    R, Q, H, _ = q.shape
    par = parent.cpu().numpy()
    out, lse = np.zeros((R, Q, H, 512)), np.full((R, Q, H), -np.inf)
    slack, zslack = np.zeros((R, Q, H, 512)), np.zeros((R, Q, H))
    for r in range(R):
        for i, path in enumerate(branches(par[r])):
            e = entry[r] if entry.dim() == 2 else entry[r, i]
            e = e[(e >= 0) & (e < rows.shape[0])].long()
            seen = torch.cat([rows[e], own[r, path]])
            at = torch.arange(len(seen), dtype=torch.int32)[None, None]
            o, z, s, zs = attend64(q[r:r + 1, i:i + 1], seen, at, scale)
            out[r, i], lse[r, i], slack[r, i], zslack[r, i] = o[0, 0], z[0, 0], s[0, 0], zs[0, 0]
    return out, lse, slack, zslack


def make_parent(R, Q, kind, rng):
    node = np.arange(Q)
    p = {"chain": np.tile(node - 1, (R, 1)), "star": np.where(node > 0, 0, -1) + np.zeros((R, 1), int),
         "apart": np.full((R, Q), -1),
         "random": np.where(node > 0, (rng.random((R, Q)) * np.maximum(node, 1)).astype(int), -1)}[kind]
    return torch.from_numpy(p.astype(np.int32)).cuda()


def tree_case(R, Q, H, K, n_rows, seed, kind="random", shared=False, pads=0.0):
    q, kv, entry, own = attend_case(R, Q, H, K, n_rows, seed, pads=pads, own=True)
    rng = np.random.default_rng(seed + 1)
    return q, kv, entry[:, 0].contiguous() if shared else entry, own, make_parent(R, Q, kind, rng)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("kind", ["random", "chain"])
@pytest.mark.parametrize("R,Q,H,K", [
    (1, 1, 1, 0), (1, 1, 16, 1), (1, 2, 5, 127), (2, 7, 20, 128), (1, 64, 3, 300), (3, 33, 4, 129), (2, 8, 64, 517),
    (1, 3, 130, 64), (1, 16, 65, 250), (40, 4, 8, 96), (2, 64, 1, 1000), (1, 5, 33, 2048)])
def test_tree(R, Q, H, K, kind, shared):
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own, parent = tree_case(R, Q, H, K, max(1, 3 * K // 2), R * 1000 + H + K, kind, shared)
    got = rows.attend_tree(q, kv, entry, SCALE, own, parent)
    check_attend(got, tree64(q, kv, entry, SCALE, own, parent))
    rows.sync()


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("kind", ["star", "apart"])
def test_tree_shapes(kind, shared):
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own, parent = tree_case(2, 40, 6, 200, 150, 3, kind, shared)
    check_attend(rows.attend_tree(q, kv, entry, SCALE, own, parent), tree64(q, kv, entry, SCALE, own, parent))


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("H", [5, 64, 100])
def test_tree_pads(H, shared):
    """Pads anywhere, lists of pads alone (a node then sees its branch), entries out of range."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own, parent = tree_case(3, 5, H, 300, 200, H, "random", shared, pads=0.3)
    entry[0] = -1
    entry[1, ..., :170] = -1
    entry[2, ..., 1::3] = 200
    entry[2, ..., 4] = torch.iinfo(torch.int32).min
    entry[2, ..., 5] = torch.iinfo(torch.int32).max
    check_attend(rows.attend_tree(q, kv, entry, SCALE, own, parent), tree64(q, kv, entry, SCALE, own, parent))


def test_tree_of_a_chain_is_attend():
    """One chain per request: ``attend`` with own rows, bit for bit."""
    from serving_step_sparse_gb300 import rows
    for R, Q, H, K in ((2, 3, 20, 300), (32, 3, 64, 500), (1, 33, 100, 129)):
        q, kv, entry, own, parent = tree_case(R, Q, H, K, 400, R, "chain", pads=0.1)
        a, b = rows.attend(q, kv, entry, SCALE, own_rows=own), rows.attend_tree(q, kv, entry, SCALE, own, parent)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_tree_parents_out_of_order():
    """A parent that is no earlier node stands for none."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own, parent = tree_case(2, 12, 9, 100, 100, 4)
    want = parent.clone()
    for i, bad in ((3, 3), (5, 11), (7, 12), (9, torch.iinfo(torch.int32).max), (11, torch.iinfo(torch.int32).min)):
        parent[:, i], want[:, i] = bad, -1
    a, b = (rows.attend_tree(q, kv, entry, SCALE, own, p) for p in (parent, want))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_attend(a, tree64(q, kv, entry, SCALE, own, parent))


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("R,Q,H,K", [(2, 9, 20, 250), (1, 40, 3, 0), (8, 4, 64, 300)])
@pytest.mark.parametrize("bad", ["codes", "scale", "inf", "rope", "negative inf"])
def test_tree_bad_own_row(R, Q, H, K, bad, shared):
    """A node's row that is not finite: NaN for the nodes that see it, nothing for the others, whose
    bits are those of a row that is."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own, parent = tree_case(R, Q, H, K, 300, Q + H, "random", shared)
    want = rows.attend_tree(q, kv, entry, SCALE, own, parent)
    node = Q // 2
    if bad == "codes":
        own[0, node, 7:500:3] = 0x7F
        own[0, node, 8:500:3] = 0xFF
    elif bad == "rope":
        own[0, node, 528:] = 0xFF
    else:
        value = {"scale": math.nan, "inf": math.inf, "negative inf": -math.inf}[bad]
        own[0, node, 516:520] = torch.tensor([value]).view(torch.uint8).cuda()
    out, lse = rows.attend_tree(q, kv, entry, SCALE, own, parent)
    for i, path in enumerate(branches(parent[0].cpu().numpy())):
        if node in path:
            assert torch.isnan(out[0, i]).all() and torch.isnan(lse[0, i]).all()
        else:
            assert torch.equal(out[0, i], want[0][0, i]) and torch.equal(lse[0, i], want[1][0, i])
    assert torch.equal(out[1:], want[0][1:]) and torch.equal(lse[1:], want[1][1:])


def test_tree_query_not_finite():
    """A node's head that is not finite leaves the others as they were."""
    from serving_step_sparse_gb300 import rows
    for shared in (False, True):
        q, kv, entry, own, parent = tree_case(1, 6, 33, 200, 200, 12, shared=shared)
        want = rows.attend_tree(q, kv, entry, SCALE, own, parent)
        q[0, 2, 5, 100], q[0, 4] = math.nan, math.inf
        out, lse = rows.attend_tree(q, kv, entry, SCALE, own, parent)
        assert torch.isnan(out[0, 2, 5]).all() and torch.isnan(out[0, 4]).all()
        same = torch.ones(6, 33, dtype=torch.bool)
        same[2, 5] = same[4] = False
        assert torch.equal(out[0][same], want[0][0][same]) and torch.equal(lse[0][same], want[1][0][same])


def test_tree_strides_and_outputs():
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own, parent = tree_case(3, 5, 12, 200, 150, 4)
    wide = torch.zeros(3, 5, 12, 640, dtype=torch.bfloat16, device="cuda")
    wide[..., 8:584] = q
    heads_first = q.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    odd = torch.zeros(3, 5, 12, 577, dtype=torch.bfloat16, device="cuda")
    odd[..., 1:] = q
    own_wide = torch.zeros(3, 7, 2, 656, dtype=torch.uint8, device="cuda")
    own_wide[:, 1:6, 1] = own
    for lists in (entry, entry[:, 0]):
        want = rows.attend_tree(q, kv, lists.contiguous(), SCALE, own, parent)
        for qq in (wide[..., 8:584], heads_first, odd[..., 1:]):
            got = rows.attend_tree(qq, kv, lists, SCALE, own_wide[:, 1:6, 1], parent.t().contiguous().t())
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        got = rows.attend_tree(q, kv, lists, SCALE, own, parent, out=out, lse=lse)
        assert got[0] is out and got[1] is lse and torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_tree_empty():
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own, parent = tree_case(2, 3, 24, 5, 4, 1)
    out, lse = rows.attend_tree(q[:0], kv, entry[:0], SCALE, own[:0], parent[:0])
    assert out.shape == (0, 3, 24, 512) and lse.shape == (0, 3, 24)
    assert rows.attend_tree(q[:, :0], kv, entry[:, :0], SCALE, own[:, :0], parent[:, :0])[0].shape == (2, 0, 24, 512)
    assert rows.attend_tree(q[:, :, :0], kv, entry, SCALE, own, parent)[0].shape == (2, 3, 0, 512)
    none = kv[:0].contiguous()
    check_attend(rows.attend_tree(q, none, entry, SCALE, own, parent), tree64(q, none, entry, SCALE, own, parent))


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("R,Q,H,K", [(90, 4, 20, 300), (60, 8, 64, 11), (7, 16, 128, 700), (160, 2, 64, 256)])
def test_tree_many_items(R, Q, H, K, shared):
    """Several items in a block, items that blocks share, many times over: the same bits."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own, parent = tree_case(R, Q, H, K, 500, R + K, "random", shared, pads=0.1)
    want = rows.attend_tree(q, kv, entry, SCALE, own, parent)
    some = slice(0, 5)
    check_attend((want[0][some], want[1][some]), tree64(q[some], kv, entry[some], SCALE, own[some], parent[some]))
    for _ in range(50):
        got = rows.attend_tree(q, kv, entry, SCALE, own, parent)
    rows.sync()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("barrier", [0, 5, 10, 11, 14, 17, 19, 20, 21])
def test_tree_gives_up(barrier):
    """A barrier that never opens: the call ends, its error is reported once, the next call is whole."""
    from serving_step_sparse_gb300 import rows, ula
    q, kv, entry, own, parent = tree_case(40, 4, 20, 300, 500, barrier)
    want = rows.attend_tree(q, kv, entry, SCALE, own, parent)
    rows.sync()
    ula.ula_rows_debug_hold(barrier)
    try:
        rows.attend_tree(q, kv, entry, SCALE, own, parent)
    finally:
        ula.ula_rows_debug_hold(-1)
    with pytest.raises(ula.UlaError) as e:
        rows.sync()
    assert e.value.code == ula.ERR_TIMEOUT
    got = rows.attend_tree(q, kv, entry, SCALE, own, parent)
    rows.sync()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------------------- score

def score64(before, q, rows, entry, address, lse, scale):
    """(scores, slack): what an address may be off by."""
    R, Q, H, _ = q.shape
    lat, rope = unpack(rows) if rows.shape[0] else (np.zeros((0, 512)), np.zeros((0, 64)))
    keys = np.concatenate([lat, rope], axis=1)
    qd, z0 = q.double().cpu().numpy(), lse.double().cpu().numpy()
    e, a = entry.cpu().numpy(), address.cpu().numpy()
    total = before.double().cpu().numpy().copy()
    slack = np.zeros_like(total)
    bits = max(3, math.ceil(math.log2(max(1, R * Q * H * e.shape[-1]))))
    for r in range(R):
        for i in range(Q):
            idx, to = (e[r], a[r]) if e.ndim == 2 else (e[r, i], a[r, i])
            ok = (idx >= 0) & (idx < rows.shape[0]) & (to >= 0) & (to < len(total))
            idx, to = idx[ok], to[ok]
            live = np.isfinite(z0[r, i])
            z = qd[r, i][live] @ keys[idx].T * scale
            err = 2.0 ** -20 * abs(scale) * (np.abs(qd[r, i][live]) @ np.abs(keys[idx]).T)
            m = z0[r, i][live][:, None]
            p = np.minimum(np.exp(z - m), 1)
            np.add.at(total, to, p.sum(0))
            loss = p * (np.expm1(err + 2.0 ** -22 * (np.abs(z) + np.abs(m))) + 2.0 ** -21)
            np.add.at(slack, to, loss.sum(0) + 2.0 ** -16 * p.sum(0) + 2.0 ** -(63 - bits) + 2.0 ** -120)
    return total, slack


def check_score(got, want):
    total, slack = want
    assert (np.abs(got.double().cpu().numpy() - total) <= slack + 2.0 ** -23 * np.abs(total) * 1.01).all()


def score_case(R, Q, H, K, n_rows, seed, pads=0.0, shared=False, n_scores=None, qscale=1.0):
    q, kv, entry, own = attend_case(R, Q, H, K, n_rows, seed, pads=pads, own=True, qscale=qscale)
    rng = np.random.default_rng(seed + 7)
    n = n_scores or 3 * n_rows + 1
    where = torch.from_numpy(rng.permutation(n)[:n_rows].astype(np.int32)).cuda()
    if shared:
        entry = entry[:, 0].contiguous()
    address = torch.where(entry >= 0, where[entry.clamp_min(0).long()], -1)
    before = torch.from_numpy(rng.random(n).astype(np.float32)).cuda()
    from serving_step_sparse_gb300 import rows
    if shared:
        wide = entry[:, None].expand(R, Q, K).contiguous()
        lse = rows.attend(q, kv, wide, SCALE)[1]
    else:
        lse = rows.attend(q, kv, entry, SCALE, own_rows=own)[1]
    return before, q, kv, entry, address, lse


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("R,Q,H,K", [
    (1, 1, 1, 1), (1, 1, 16, 127), (1, 2, 17, 128), (2, 3, 32, 129), (1, 2, 33, 255), (3, 1, 64, 256), (1, 1, 65, 300),
    (2, 2, 128, 517), (1, 1, 130, 64), (1, 4, 20, 2048), (40, 1, 8, 96), (1, 8, 128, 200), (3, 5, 100, 140),
    (1, 1, 257, 130), (2, 33, 7, 50)])
def test_score(R, Q, H, K, shared):
    from serving_step_sparse_gb300 import rows
    before, *case = score_case(R, Q, H, K, max(1, 2 * K // 3), R * 100 + H + K, shared=shared)
    scores = before.clone()
    assert rows.score(scores, *case, SCALE) is scores
    rows.sync()
    check_score(scores, score64(before, *case, SCALE))


@pytest.mark.parametrize("H", [5, 64, 100])
def test_score_pads(H):
    """Pads, whole tiles and lists of pads, rows and addresses out of range, tokens and heads without an lse."""
    from serving_step_sparse_gb300 import rows
    before, q, kv, entry, address, lse = score_case(3, 2, H, 700, 500, H, pads=0.3)
    entry[0, 0] = -1
    entry[0, 1, :400] = -1
    entry[1, 0, ::2] = torch.iinfo(torch.int32).min
    entry[1, 1, 1::3] = 500
    address[2, 0, ::5] = len(before)
    address[2, 0, 1::5] = -1
    address[2, 0, 2::5] = torch.iinfo(torch.int32).max
    address[2, 0, 3] = torch.iinfo(torch.int32).min
    lse[1, 1, H // 2] = -math.inf
    lse[2, 1] = -math.inf
    scores = before.clone()
    rows.score(scores, q, kv, entry, address, lse, SCALE)
    check_score(scores, score64(before, q, kv, entry, address, lse, SCALE))
    named = torch.zeros(len(before), dtype=torch.bool, device="cuda")
    named[address[(address >= 0) & (address < len(before))].long()] = True
    assert torch.equal(scores[~named], before[~named])       # nothing beside the addresses that are named


def test_score_repeated_addresses():
    """The same address many times, in one list and in several: every weight counts, in any order."""
    from serving_step_sparse_gb300 import rows
    before, q, kv, entry, address, lse = score_case(2, 3, 40, 900, 600, 5)
    address %= 7
    want = score64(before, q, kv, entry, address, lse, SCALE)
    scores = before.clone()
    rows.score(scores, q, kv, entry, address, lse, SCALE)
    check_score(scores, want)
    for _ in range(10):
        again = before.clone()
        rows.score(again, q, kv, entry, address, lse, SCALE)
        assert torch.equal(again, scores)
    turn = torch.randperm(900, device="cuda")
    again = before.clone()
    rows.score(again, q, kv, entry[..., turn].contiguous(), address[..., turn].contiguous(), lse, SCALE)
    assert torch.equal(again, scores)


def test_score_sums_to_the_heads():
    """The weights of a token's whole list are one for each head."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, _ = attend_case(3, 2, 48, 1000, 800, 3, qscale=4.0)
    lse = rows.attend(q, kv, entry, SCALE)[1]
    address = (torch.arange(6, device="cuda", dtype=torch.int32).view(3, 2, 1)).expand(3, 2, 1000).contiguous()
    scores = rows.score(torch.zeros(6, device="cuda"), q, kv, entry, address, lse, SCALE)
    assert (scores - 48).abs().max() <= 48 * 2.0 ** -12


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_score_not_finite(bad):
    """Weights that are no numbers count for nothing; a weight is 1 at most."""
    from serving_step_sparse_gb300 import rows
    before, q, kv, entry, address, lse = score_case(1, 3, 33, 260, 300, 21)
    want = score64(before, q[:, 1:], kv, entry[:, 1:], address[:, 1:], lse[:, 1:], SCALE)
    scores = before.clone()
    broken, none = q.clone(), lse.clone()
    broken[0, 0] = bad
    none[0, 0] = bad
    if bad != math.inf:
        rows.score(scores, broken, kv, entry, address, none, SCALE)
        check_score(scores, want)
    scores = before.clone()
    none = lse.clone()
    none[0, 0] = bad if bad != -math.inf else math.nan      # of a token whose queries are numbers
    rows.score(scores, q, kv, entry, address, none, SCALE)
    check_score(scores, want)
    scores = before.clone()
    none = lse.clone()
    none[0, 1] = -1000.0                                     # (an lse that does not fit)
    rows.score(scores, q, kv, entry, address, none, SCALE)
    check_score(scores, score64(before, q, kv, entry, address, none, SCALE))
    rotten = kv.clone()
    rotten[299, :512] = 0x7F                                 # a row that no list holds, one that a list does
    rotten[298, 512:516] = torch.tensor([bad]).view(torch.uint8).cuda()
    entry = entry.clamp_max(297)
    scores, clean = before.clone(), before.clone()
    rows.score(clean, q, kv, entry, address, lse, SCALE)
    rows.score(scores, q, rotten, entry, address, lse, SCALE)
    assert torch.equal(scores, clean)
    entry[0, 2, 100], address[0, 2, 100] = 299, 5
    at = torch.arange(len(before), device="cuda") != 5
    rows.score(clean.copy_(before), q, kv, entry, address, lse, SCALE)
    rows.score(scores.copy_(before), q, rotten, entry, address, lse, SCALE)
    assert torch.equal(scores[at], clean[at]) and torch.isfinite(scores).all()


def test_score_strides():
    from serving_step_sparse_gb300 import rows
    before, q, kv, entry, address, lse = score_case(3, 2, 12, 200, 150, 4)
    want = rows.score(before.clone(), q, kv, entry, address, lse, SCALE)
    wide = torch.zeros(3, 2, 12, 640, dtype=torch.bfloat16, device="cuda")
    wide[..., 8:584] = q
    heads_first = q.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    odd = torch.zeros(3, 2, 12, 577, dtype=torch.bfloat16, device="cuda")
    odd[..., 1:] = q
    back = lambda t: t.permute(2, 1, 0).contiguous().permute(2, 1, 0)  # noqa: E731
    for qq in (wide[..., 8:584], heads_first, odd[..., 1:]):
        assert torch.equal(rows.score(before.clone(), qq, kv, back(entry), back(address), back(lse), SCALE), want)


def test_score_far_rows():
    """A gathered buffer past 2^32 bytes, and scores whose sums lie past 2^32 bytes."""
    from serving_step_sparse_gb300 import rows
    n = 2 ** 32 // 656 + 1000
    big = torch.zeros(n, 656, dtype=torch.uint8, device="cuda")
    before, q, kv, entry, address, lse = score_case(1, 1, 16, 300, 300, 6)
    big[-300:] = kv
    want = rows.score(before.clone(), q, kv, entry, address, lse, SCALE)
    far = torch.zeros(2 ** 29 + 5000, device="cuda")
    far[-len(before):] = before
    got = rows.score(far, q, big, entry + (n - 300), address + (len(far) - len(before)), lse, SCALE)
    assert torch.equal(got[-len(before):], want) and not got[:-len(before)].any()


def test_score_empty():
    from serving_step_sparse_gb300 import rows
    before, q, kv, entry, address, lse = score_case(2, 3, 24, 5, 4, 1)
    for args in ((q[:0], kv, entry[:0], address[:0], lse[:0]), (q[:, :0], kv, entry[:, :0], address[:, :0], lse[:, :0]),
                 (q[:, :, :0], kv, entry, address, lse[:, :, :0]), (q, kv, entry[..., :0], address[..., :0], lse),
                 (q, kv[:0].contiguous(), entry, address, lse)):
        assert torch.equal(rows.score(before.clone(), *args, SCALE), before)
    assert rows.score(before[:0], q, kv, entry, address, lse, SCALE).shape == (0,)


def test_score_two_calls_at_once():
    """Calls on streams of their own that update the same scores: nothing is lost."""
    from serving_step_sparse_gb300 import rows
    before, *case = score_case(8, 2, 40, 600, 500, 9)
    streams = [torch.cuda.Stream() for _ in range(3)]
    scores = torch.zeros_like(before)
    one = rows.score(torch.zeros_like(before), *case, SCALE)
    torch.cuda.synchronize()
    for _ in range(4):
        for s in streams:
            rows.score(scores, *case, SCALE, stream=s)
    torch.cuda.synchronize()
    # 12 additions in fp32 of the same number
    assert ((scores - 12 * one).abs() <= 12 * 2.0 ** -23 * 12 * one.abs()).all()


@pytest.mark.parametrize("R,Q,H,K", [(220, 1, 64, 11), (55, 2, 129, 130), (400, 1, 3, 100), (90, 2, 20, 300), (16, 3, 128, 2048)])
def test_score_many_items(R, Q, H, K):
    """Many lists per block, many times over: the same bits."""
    from serving_step_sparse_gb300 import rows
    before, *case = score_case(R, Q, H, K, 500, R + K, pads=0.1)
    want = rows.score(before.clone(), *case, SCALE)
    check_score(want, score64(before, *case, SCALE))
    for _ in range(50):
        got = rows.score(before.clone(), *case, SCALE)
    rows.sync()
    assert torch.equal(got, want)


# ------------------------------------------------------------------------------- evict

def evict_lists(scores, address, length, budget, first, last):
    s, a, n_of = scores.cpu().numpy(), address.cpu().numpy(), length.cpu().numpy()
    R, N = a.shape
    kept, dropped = np.full((R, budget), -1, np.int32), np.full((R, max(0, N - budget)), -1, np.int32)
    for r in range(R):
        n = min(max(int(n_of[r]), 0), N)
        at = a[r, :n].astype(np.int64)
        inside = (at >= 0) & (at < len(s))
        v = np.where(inside, s[np.where(inside, at, 0)] if len(s) else 0, np.float32(0)).astype(np.float64)
        drop = np.zeros(n, bool)
        if n > budget:
            mid = np.arange(first, n - last)
            order = np.lexsort((mid, np.where(np.isnan(v[mid]), 0, v[mid]), np.isnan(v[mid])))
            drop[mid[order[:n - budget]]] = True
        kept[r, :n - drop.sum()], dropped[r, :drop.sum()] = a[r, :n][~drop], a[r, :n][drop]
    return kept, dropped


def check_evict(scores, address, length, budget, first=0, last=0):
    from serving_step_sparse_gb300 import rows
    got = rows.evict(scores, address, length, budget, first=first, last=last)
    want = evict_lists(scores, address, length, budget, first, last)
    assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])


def evict_case(R, N, n_scores, seed, kind):
    rng = np.random.default_rng(seed)
    s = {"any": rng.standard_normal(n_scores), "unused": np.where(rng.random(n_scores) < 0.7, 0, rng.random(n_scores) ** 4),
         "few": rng.integers(-2, 3, n_scores) * 0.5, "equal": np.full(n_scores, 0.25),
         "close": 1 + rng.integers(0, 5, n_scores) * 2.0 ** -23,
         "wide": rng.standard_normal(n_scores) * 10.0 ** rng.integers(-44, 38, n_scores)}[kind].astype(np.float32)
    address = rng.integers(0, n_scores, (R, N)).astype(np.int32)
    length = rng.integers(0, N + 1, R).astype(np.int32)
    length[rng.integers(0, R)] = N
    return torch.from_numpy(s).cuda(), torch.from_numpy(address).cuda(), torch.from_numpy(length).cuda()


@pytest.mark.parametrize("kind", ["any", "unused", "few", "equal", "close", "wide"])
@pytest.mark.parametrize("R,N", [(1, 1), (3, 31), (2, 32), (5, 33), (2, 511), (4, 1000), (1, 2048), (3, 2049), (2, 5000),
                                 (1, 16384), (2, 16385), (3, 40000)])
def test_evict(R, N, kind):
    case = evict_case(R, N, N + 7, R + N, kind)
    for budget, first, last in ((0, 0, 0), (1, 0, 1), (N // 3, 0, 0), (N // 2, N // 8, N // 4), (N - 1, 0, 0), (N, 0, 0), (N + 5, 2, 3),
                                (N // 2, N // 2 - N // 4, N // 4)):
        check_evict(*case, budget, first, last)


@pytest.mark.parametrize("kind", ["any", "unused", "equal"])
@pytest.mark.parametrize("R,N,budget", [(1, 131072, 40000), (5, 100001, 99999), (2, 393217, 150000), (1, 700000, 3), (300, 700, 100)])
def test_evict_long(R, N, budget, kind):
    """Lists over several blocks, longer than the blocks' keys in shared memory, many requests."""
    case = evict_case(R, N, N, R + N, kind)
    check_evict(*case, budget)
    check_evict(*case, budget, budget // 3, budget // 2)


def test_evict_values():
    """NaN, infinities, zeros of both signs, subnormals; addresses out of range; lengths out of range."""
    rng = np.random.default_rng(2)
    odd = np.array([math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-45, -1e-45, 3e38, -3e38, 1.0], np.float32)
    scores = torch.from_numpy(rng.choice(odd, 500)).cuda()
    scores[::17] = torch.tensor(-math.nan)
    address = torch.from_numpy(rng.integers(-3, 520, (4, 900)).astype(np.int32)).cuda()
    address[1, :5] = torch.tensor([2 ** 31 - 1, -2 ** 31, 500, 499, -1], device="cuda")
    length = torch.tensor([900, 901, -5, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    for budget in (0, 1, 100, 450, 640, 899):
        check_evict(scores, address, length, budget)
        check_evict(scores, address, length, budget, budget // 2, budget // 2)
    check_evict(scores[:0], address, length, 300)


def test_evict_empty_and_outputs():
    from serving_step_sparse_gb300 import rows
    scores, address, length = evict_case(3, 100, 100, 1, "any")
    kept, dropped = rows.evict(scores, address[:0], length[:0], 10)
    assert kept.shape == (0, 10) and dropped.shape == (0, 90)
    kept, dropped = rows.evict(scores, address[:, :0], length, 10)
    assert (kept == -1).all() and dropped.shape == (3, 0)
    want = rows.evict(scores, address, length, 30, first=2, last=3)
    kept, dropped = torch.empty_like(want[0]), torch.empty_like(want[1])
    got = rows.evict(scores, address, length, 30, first=2, last=3, kept=kept, dropped=dropped)
    assert got[0] is kept and got[1] is dropped and torch.equal(kept, want[0]) and torch.equal(dropped, want[1])
    spread = torch.zeros(200, device="cuda")
    spread[::2] = scores
    got = rows.evict(spread[::2], address.t().contiguous().t(), length, 30, first=2, last=3)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------------------- norm and rotate

def normed(x, weight, eps):
    x, w = x.double().cpu().numpy(), weight.double().cpu().numpy()
    with np.errstate(invalid="ignore", divide="ignore"):
        return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def check_norm(got, x, weight, eps, at, pos, freq, axis, pairing, dtype):
    want = normed(x, weight, eps)
    slack = np.abs(want).copy()
    want[..., at:at + 64], length = turned(want[..., at:at + 64], pos, freq, axis, pairing)
    slack[..., at:at + 64] = 1.5 * length      # (a turned value is of two normed ones: at most sqrt(2) of their length)
    tol = HALF_ULP[dtype] * np.abs(want) * 1.01 + (NORM + 2.0 ** -20) * slack + SMALLEST[dtype]
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(want))
    ok = ~np.isnan(want)
    assert (np.abs(g - want) <= tol)[ok].all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,heads,width,at", [
    (1, 1, 64, 0), (3, 5, 128, 64), (3, 5, 128, 0), (17, 64, 192, 128), (33, 3, 96, 32), (9, 7, 200, 136), (5, 2, 201, 130), (11, 4, 65, 1),
    (700, 1, 64, 0), (33, 128, 256, 192), (6, 10, 576, 512), (4, 3, 1024, 480), (4, 3, 1023, 5), (2, 6, 640, 576), (5, 5, 384, 104)])
def test_norm_rotate(n, heads, width, at, dtype):
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(n * 131 + heads + width)
    x = torch.from_numpy(rng.standard_normal((n, heads, width)) * np.exp(2 * rng.standard_normal((n, heads, 1)))).to(DT[dtype]).cuda()
    pos = positions(rng, 3, n)
    pos_d = torch.from_numpy(pos).cuda()
    for pairing in ("adjacent", "halves"):
        rot, freq, axis = make_rotary(rng, 3, pairing)
        for wt in {dtype, "f32"}:
            w = torch.from_numpy(1 + 0.3 * rng.standard_normal(width)).to(DT[wt]).cuda()
            out = rows.norm_rotate(x, w, pos_d, rot, at=at)
            check_norm(out, x, w, 1e-6, at, pos, freq, axis, pairing, dtype)
            y = x.clone()
            assert rows.norm_rotate(y, w, pos_d, rot, at=at, out=y) is y and torch.equal(y, out)     # in place
            if at == width - 64:
                assert torch.equal(rows.norm_rotate(x, w, pos_d, rot), out)
        out = rows.norm_rotate(x, w, pos_d, rot, at=at, eps=0.5)
        check_norm(out, x, w, 0.5, at, pos, freq, axis, pairing, dtype)
        assert torch.equal(rows.norm_rotate(x[:, 0], w, pos_d, rot, at=at, eps=0.5), out[:, 0])      # no head axis


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset,head_stride,token_extra", [(0, 192, 0), (64, 576, 0), (8, 208, 16), (1, 193, 3), (2, 194, 2), (64, 576, 1)])
def test_norm_strides_and_alignment(dtype, offset, head_stride, token_extra):
    """The same bits whatever the alignment; nothing beside the heads is touched."""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(offset + head_stride)
    n, heads, width, at = 37, 6, 192, 128
    rot, freq, axis = make_rotary(rng, 3, "halves")
    store = torch.from_numpy(rng.standard_normal(offset + n * (heads * head_stride + token_extra) + width)).to(DT[dtype]).cuda()
    view = store.as_strided((n, heads, width), (heads * head_stride + token_extra, head_stride, 1), offset)
    x = view.clone()
    w = torch.from_numpy(rng.random(width) + 0.5).to(DT[dtype]).cuda()
    pos = positions(rng, 5, n)
    pos_d = torch.from_numpy(pos).cuda()
    dense = rows.norm_rotate(view, w, pos_d, rot)
    check_norm(dense, x, w, 1e-6, at, pos, freq, axis, "halves", dtype)
    before = store.clone()
    rows.norm_rotate(view, w, pos_d, rot, out=view)
    assert torch.equal(view, dense)
    mask = torch.ones_like(store, dtype=torch.bool)
    mask.as_strided(view.shape, view.stride(), offset).fill_(False)
    assert torch.equal(store[mask], before[mask])
    odd = torch.zeros(width + 1, dtype=w.dtype, device="cuda")
    odd[1:] = w
    assert torch.equal(rows.norm_rotate(x, odd[1:], pos_d, rot), dense)
    assert torch.equal(rows.norm_rotate(x, w.repeat_interleave(2)[::2], pos_d, rot), dense)
    assert torch.equal(rows.norm_rotate(x.transpose(1, 2).contiguous().transpose(1, 2), w, pos_d, rot), dense)


def test_norm_values():
    """Zeros (with eps and without), NaN and infinities stay within their head."""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(4)
    rot, freq, axis = make_rotary(rng, 2, "adjacent")
    pos = positions(rng, 2, 4)
    pos_d = torch.from_numpy(pos).cuda()
    for dtype in DT:
        for width in (128, 130):
            x = torch.from_numpy(rng.standard_normal((4, 5, width))).to(DT[dtype]).cuda()
            w = torch.ones(width, device="cuda")
            x[0, 1] = 0
            for eps in (0.0, 1e-6):
                out = rows.norm_rotate(x, w, pos_d, rot, eps=eps)
                check_norm(out, x, w, eps, width - 64, pos, freq, axis, "adjacent", dtype)
            clean = rows.norm_rotate(x, w, pos_d, rot)
            x[1, 2, 3], x[2, 0, 70], x[3, 4, width - 1] = math.nan, math.inf, -math.inf
            out = rows.norm_rotate(x, w, pos_d, rot)
            bad = torch.zeros(4, 5, dtype=torch.bool, device="cuda")
            bad[1, 2] = bad[2, 0] = bad[3, 4] = True
            assert torch.equal(out[~bad], clean[~bad]) and torch.isnan(out[1, 2]).all()
            assert torch.isnan(out[2, 0, 70]) and torch.isnan(out[3, 4, width - 1])


def test_norm_many():
    """More rows than the GPU holds at once, of few and of many heads; the rotation alone beside it."""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(6)
    for n, heads, width in ((40001, 1, 128), (700, 131, 192), (3001, 9, 64)):
        rot, freq, axis = make_rotary(rng, 2, "halves")
        x = torch.from_numpy(rng.standard_normal((n, heads, width)).astype(np.float32)).to(torch.bfloat16).cuda()
        w = torch.from_numpy(rng.random(width) + 0.5).float().cuda()
        pos = positions(rng, 2, n)
        out = rows.norm_rotate(x, w, torch.from_numpy(pos).cuda(), rot)
        check_norm(out, x, w, 1e-6, width - 64, pos, freq, axis, "halves", "bf16")


# ------------------------------------------------------------------------------- norm and pack

def check_pack_norm(got, latent, rope, w, rw, eps, pos, freq, axis, pairing):
    n = latent.shape[0]
    b = got.cpu().numpy()
    v = normed(latent, w, eps).reshape(n, 4, 128)
    scale = np.ascontiguousarray(b[:, 512:528]).view(np.float32).astype(np.float64)
    want = np.maximum(np.abs(v).max(-1) / 448, 2.0 ** -126)
    assert (np.abs(scale - want) <= (NORM + 2.0 ** -23) * want).all()
    codes = E4M3[b[:, :512]].reshape(n, 4, 128)
    y = v / scale[..., None]
    spacing = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    assert (np.abs(codes - y) <= spacing / 2 + (NORM + 2.0 ** -20) * np.abs(y)).all()
    rn = rope.double().cpu().numpy() if rw is None else normed(rope, rw, eps)
    rn, length = turned(rn, pos, freq, axis, pairing)
    bits = np.ascontiguousarray(b[:, 528:]).view(np.uint16).astype(np.uint32) << 16
    tol = 2.0 ** -8 * np.abs(rn) * 1.01 + (2.0 ** -20 + (0 if rw is None else 1.5 * NORM)) * length + 2.0 ** -133
    assert (np.abs(bits.view(np.float32) - rn) <= tol).all()


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,layers", [(1, 1), (7, 4), (8, 1), (129, 3), (1000, 1), (5000, 2)])
def test_pack_norm(n, layers, dtype, pairing):
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(n * 7 + layers)
    rot, freq, axis = make_rotary(rng, 3, pairing)
    x = rng.standard_normal((n, 512)) * np.exp(rng.standard_normal((n, 1)))
    x[0, :128] = 0
    x[n // 2, 128:256] *= 1e-4
    x[n - 1, 384:] *= 50
    latent = torch.from_numpy(x).to(DT[dtype]).cuda()
    rope = torch.from_numpy(3 * rng.standard_normal((n, 64))).to(DT[dtype]).cuda()
    pos = positions(rng, 3, n)
    pos_d = torch.from_numpy(pos).cuda()
    for wt in {dtype, "f32"}:
        w = torch.from_numpy(1 + 0.3 * rng.standard_normal(512)).to(DT[wt]).cuda()
        for rw in (None, torch.from_numpy(1 + 0.3 * rng.standard_normal(64)).to(DT[wt]).cuda()):
            dest = torch.full((n, layers, 656), 0xA5, dtype=torch.uint8, device="cuda")
            got = rows.pack_norm(latent, rope, w, pos_d, rot, dest[:, layers - 1], rope_weight=rw)
            assert got.data_ptr() == dest[:, layers - 1].data_ptr() and (dest[:, :layers - 1] == 0xA5).all()
            check_pack_norm(got, latent, rope, w, rw, 1e-6, pos, freq, axis, pairing)
            assert torch.equal(rows.pack_norm(latent, rope, w, pos_d, rot, rope_weight=rw), got)
    got = rows.pack_norm(latent, rope, w, pos_d, rot, rope_weight=rw, eps=2.0)
    check_pack_norm(got, latent, rope, w, rw, 2.0, pos, freq, axis, pairing)


def test_pack_norm_strides_and_values():
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(5)
    rot, _, _ = make_rotary(rng, 2, "adjacent")
    n = 21
    for dtype in DT.values():
        wide = torch.from_numpy(rng.standard_normal((n, 600))).to(dtype).cuda()
        pos = torch.from_numpy(positions(rng, 2, n)).cuda()
        w, rw = wide[0, :512].clone(), wide[1, :64].clone()
        for at in (0, 1, 8, 13):
            latent, rope = wide[:, at:at + 512], wide[:, at + 513:at + 577]
            want = rows.pack_norm(latent.contiguous(), rope.contiguous(), w, pos, rot, rope_weight=rw)
            assert torch.equal(rows.pack_norm(latent, rope, w.repeat_interleave(2)[::2], pos, rot, rope_weight=rw), want)
    latent = torch.ones(3, 512, device="cuda")
    rope = torch.ones(3, 64, device="cuda")
    latent[1, 200], rope[2, 9] = math.nan, math.inf
    got = rows.pack_norm(latent, rope, torch.ones(512, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"),
                         rows.Rotary([0.0] * 32), rope_weight=torch.ones(64, device="cuda"))
    lat, rp = unpack(got)
    assert np.isnan(lat[1]).all() and np.isfinite(lat[[0, 2]]).all()
    assert np.isfinite(rp[:2]).all() and np.isnan(rp[2, 9])


# ------------------------------------------------------------------------------- refusals

def test_refusals():
    from serving_step_sparse_gb300 import rows, ula
    q, kv, entry, own, parent = tree_case(2, 3, 8, 16, 16, 1)
    address, lse, scores = entry.clone(), torch.zeros(2, 3, 8, device="cuda"), torch.zeros(20, device="cuda")
    length = torch.zeros(2, dtype=torch.int32, device="cuda")
    pos = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    rot = rows.Rotary([1.0] * 32)
    x, w = torch.zeros(4, 8, 128, device="cuda"), torch.ones(128, device="cuda")
    lat, rp, lw = torch.zeros(4, 512, device="cuda"), torch.zeros(4, 64, device="cuda"), torch.ones(512, device="cuda")
    many = torch.zeros(2, 65, 8, 576, dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: rows.attend_tree(q, kv, entry, SCALE, None, parent),
        lambda: rows.attend_tree(q, kv, entry, SCALE, own[:1], parent),
        lambda: rows.attend_tree(q, kv, entry, SCALE, own, parent[:1]),
        lambda: rows.attend_tree(q, kv, entry, SCALE, own, parent.long()),
        lambda: rows.attend_tree(q, kv, entry, SCALE, own, parent[0]),
        lambda: rows.attend_tree(q, kv, entry, SCALE, own, parent.cpu()),
        lambda: rows.attend_tree(q, kv, entry[0], SCALE, own, parent),
        lambda: rows.attend_tree(q, kv, entry[:, :2], SCALE, own, parent),
        lambda: rows.attend_tree(q.float(), kv, entry, SCALE, own, parent),
        lambda: rows.attend_tree(many, kv, entry[:, 0], SCALE, torch.zeros(2, 65, 656, dtype=torch.uint8, device="cuda"),
                                 torch.zeros(2, 65, dtype=torch.int32, device="cuda")),
        lambda: rows.attend(q, kv, entry[:, 0], SCALE),
        lambda: rows.score(scores.double(), q, kv, entry, address, lse, SCALE),
        lambda: rows.score(scores.view(4, 5), q, kv, entry, address, lse, SCALE),
        lambda: rows.score(scores[::2], q, kv, entry, address, lse, SCALE),
        lambda: rows.score(scores.cpu(), q, kv, entry, address, lse, SCALE),
        lambda: rows.score(scores, q, kv, entry, address.long(), lse, SCALE),
        lambda: rows.score(scores, q, kv, entry, address[..., :3], lse, SCALE),
        lambda: rows.score(scores, q, kv, entry[:, :2], address[:, :2], lse, SCALE),
        lambda: rows.score(scores, q, kv, entry, address, lse[..., :3], SCALE),
        lambda: rows.score(scores, q, kv, entry, address, lse.half(), SCALE),
        lambda: rows.score(scores, q, kv[::2], entry, address, lse, SCALE),
        lambda: rows.evict(scores.half(), address[:, 0], length, 4),
        lambda: rows.evict(scores, address, length, 4),
        lambda: rows.evict(scores, address[:, 0].long(), length, 4),
        lambda: rows.evict(scores, address[:, 0], length[:1], 4),
        lambda: rows.evict(scores, address[:, 0], length.long(), 4),
        lambda: rows.evict(scores, address[:, 0], length, -1),
        lambda: rows.evict(scores, address[:, 0], length, 4, first=3, last=2),
        lambda: rows.evict(scores, address[:, 0], length, 4, first=-1),
        lambda: rows.evict(scores, address[:, 0], length, 2 ** 31),
        lambda: rows.evict(scores, address[:, 0], length, 4, kept=torch.zeros(2, 5, dtype=torch.int32, device="cuda")),
        lambda: rows.evict(scores, address[:, 0], length, 4, dropped=torch.zeros(2, 16, dtype=torch.int32, device="cuda")),
        lambda: rows.evict(scores, address[:, 0].cpu(), length, 4),
        lambda: rows.norm_rotate(x[..., :63], w[:63], pos, rot),
        lambda: rows.norm_rotate(torch.zeros(4, 1025, device="cuda"), torch.ones(1025, device="cuda"), pos, rot),
        lambda: rows.norm_rotate(x, w[:127], pos, rot),
        lambda: rows.norm_rotate(x, w.half(), pos, rot),
        lambda: rows.norm_rotate(x.double(), w, pos, rot),
        lambda: rows.norm_rotate(x, w, pos[:, :3], rot),
        lambda: rows.norm_rotate(x, w, pos, rot, at=65),
        lambda: rows.norm_rotate(x, w, pos, rot, at=-1),
        lambda: rows.norm_rotate(x, w, pos, rot, eps=-1.0),
        lambda: rows.norm_rotate(x, w, pos, rot, eps=math.nan),
        lambda: rows.norm_rotate(x, w, pos, rot, eps=math.inf),
        lambda: rows.norm_rotate(x, w, pos, rot, out=x.half()),
        lambda: rows.norm_rotate(x.clone().requires_grad_(), w, pos, rot),
        lambda: rows.norm_rotate(x, w.clone().requires_grad_(), pos, rot),
        lambda: rows.pack_norm(lat, rp, lw[:64], pos, rot),
        lambda: rows.pack_norm(lat, rp, lw.half(), pos, rot),
        lambda: rows.pack_norm(lat, rp, lw, pos, rot, rope_weight=lw),
        lambda: rows.pack_norm(lat, rp, lw, pos, rot, eps=-1e-6),
        lambda: rows.pack_norm(lat, rp.half(), lw, pos, rot),
        lambda: rows.pack_norm(lat, rp, lw.cpu(), pos, rot),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {i} was accepted")
    store = torch.zeros(4 * 656 + 64, dtype=torch.uint8, device="cuda")
    for f in (lambda: rows.attend_tree(q, store[8:8 + 3 * 656].view(3, 656), entry, SCALE, own, parent),
              lambda: rows.score(scores, q, store[8:8 + 3 * 656].view(3, 656), entry, address, lse, SCALE),
              lambda: rows.norm_rotate(x, w, pos, rot, out=x[:1].expand(4, 8, 128)),
              lambda: rows.norm_rotate(x, w, pos, rows.Rotary([math.nan] + [1.0] * 31)),
              lambda: rows.pack_norm(lat, rp, lw, pos, rot, store[8:8 + 4 * 656].view(4, 656))):
        with pytest.raises(ula.UlaError) as e:
            f()
        assert e.value.code == ula.ERR_INVALID_ARG
    rows.sync()


# ------------------------------------------------------------------------------- together

@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("R,Q,H,K", [(3, 4, 20, 300), (33, 3, 64, 500)])
def test_a_step_in_a_graph(R, Q, H, K, shared):
    """A layer's calls of a drafted step (queries and keys normed and turned, the tree's attention, the
    weights accumulated, addresses evicted) captured once and replayed on new inputs."""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(R)
    rot, _, _ = make_rotary(rng, 1, "halves")
    pos = torch.arange(R * Q, dtype=torch.int32, device="cuda")
    w = torch.from_numpy(rng.random(576) + 0.5).to(torch.bfloat16).cuda()
    n = 400
    length = torch.full((1,), n, dtype=torch.int32, device="cuda")
    every = torch.arange(n, dtype=torch.int32, device="cuda")[None]
    cases = [tree_case(R, Q, H, K, n, 70 + s, shared=shared, pads=0.1) for s in range(3)]
    new = [torch.from_numpy(rng.standard_normal((R * Q, 576))).to(torch.bfloat16).cuda() for s in range(3)]

    def layer(q, kv, entry, parent, x, scores):
        turned_q = rows.norm_rotate(q.view(R * Q, H, 576), w, pos, rot).view(R, Q, H, 576)
        own = rows.pack_norm(x[:, :512], x[:, 512:], w[:512], pos, rot, rope_weight=w[:64]).view(R, Q, 656)
        out, lse = rows.attend_tree(turned_q, kv, entry, SCALE, own, parent)
        rows.score(scores, turned_q, kv, entry, entry, lse, SCALE)
        return (out, lse, scores, *rows.evict(scores, every, length, 100, first=4, last=16))

    def inputs(s):
        q, kv, entry, _, parent = cases[s]
        return [q, kv, entry, parent, new[s], torch.zeros(n, device="cuda")]

    want = [layer(*inputs(s)) for s in range(3)]
    held = [t.clone() for t in inputs(0)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(*held)
    for s in (1, 2, 0, 1):
        for h, t in zip(held, inputs(s)):
            h.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for g, x in zip(got, want[s]):
            assert torch.equal(g, x)
    rows.sync()


def test_other_streams():
    """Calls on streams of their own: inputs and temporaries are held until they have run."""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(3)
    rot, _, _ = make_rotary(rng, 1, "halves")
    streams = [torch.cuda.Stream() for _ in range(3)]
    cases = [tree_case(2, 5, 40, 600, 500, 30 + s) for s in range(3)]
    pos = torch.arange(10, dtype=torch.int32, device="cuda")
    w = torch.ones(576, dtype=torch.bfloat16, device="cuda")

    def chain(q, kv, entry, own, parent, stream=None):
        odd = torch.zeros(*q.shape[:3], 577, dtype=torch.bfloat16, device="cuda")
        odd[..., 1:] = q
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        y = rows.norm_rotate(odd.view(10, 40, 577)[..., 1:], w, pos, rot, stream=stream)
        out, lse = rows.attend_tree(y.view(2, 5, 40, 576), kv, entry, SCALE, own, parent, stream=stream)
        scores = torch.zeros(500, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        rows.score(scores, y.view(2, 5, 40, 576), kv, entry, entry, lse, SCALE, stream=stream)
        return out, lse, scores

    want = [chain(*c) for c in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, c in zip(streams, cases):
            got.append(chain(*c, stream=s))
            torch.zeros(2, 5, 40, 577, dtype=torch.bfloat16, device="cuda").fill_(7.0)
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for x, y in zip(g, want[i % 3]):
            assert torch.equal(x, y)


@pytest.mark.parametrize("R,Q,H,K,barrier", [(60, 2, 100, 500, b) for b in range(44)] + [
    (*c, b) for c in ((90, 1, 20, 300), (3, 2, 64, 700)) for b in (0, 4, 8, 12, 16, 20, 28, 32, 37, 42)])
def test_score_gives_up(R, Q, H, K, barrier):
    """A barrier that never opens: the call ends, its error, if somebody waited for it, is reported once, and
    the next call is whole.  (Blocks of one tile, or two, do not wait for a second phase of anything; the last
    case's blocks have several tiles, of several items.)"""
    from serving_step_sparse_gb300 import rows, ula
    before, *case = score_case(R, Q, H, K, 500, barrier)
    want = rows.score(before.clone(), *case, SCALE)
    rows.sync()
    ula.ula_rows_debug_hold_score(barrier)
    try:
        rows.score(before.clone(), *case, SCALE)
    finally:
        ula.ula_rows_debug_hold_score(-1)
    # full and empty stages (two of four with 128 columns), accumulators (three of four), the places of four tiles,
    # queries, the end
    always = [0, 1, 8, 9, 10, 16, 20, 28, 32, 33, 34, 35, 36, 42, 43]
    if barrier in always or (H == 100 and barrier in (4, 5, 12, 13, 14, 37, 38, 39, 40, 41)):
        with pytest.raises(ula.UlaError) as e:
            rows.sync()
        assert e.value.code == ula.ERR_TIMEOUT
    else:
        try:
            rows.sync()
        except ula.UlaError as e:
            assert e.code == ula.ERR_TIMEOUT
    rows.sync()
    got = rows.score(before.clone(), *case, SCALE)
    rows.sync()
    assert torch.equal(got, want)


def test_draft_tree_example():
    """The operators with the cache, as drafted steps use them, against a dense computation in 64 bits.
    Outputs are averages of normed latents (at most 6 * 1.5, a weight's spread included): rounded to bf16, with
    the probabilities' 2^-8: off by at most 2 * 2^-8 * 9.  An address's score is a sum of at most
    steps * nodes * layers * groups * heads weights of at most 1, each off by less than 2^-14 of itself (a
    logit's error is below 2^-20 * 576 * 9 * 9 * scale), added up in 32 additions in fp32."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_tree.py")
    spec = importlib.util.spec_from_file_location("draft_tree", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    steps = 3
    err, off = example.run(steps=steps, seed=1, check=True)
    most = steps * example.NODES * example.LAYERS * example.GROUPS * example.HEADS
    assert err <= 2 * 2.0 ** -8 * 9
    assert off <= most * 2.0 ** -10


def test_free_each():
    """What evict drops goes to the cache in any order; the rest stays."""
    from serving_step_sparse_gb300 import ula
    from serving_step_sparse_gb300.cache import UlaCache
    cache = UlaCache(row_bytes=16, layers_per_group=[1], gpu_slots=40, host_slots=40, ring_buckets=2, max_logical=100, max_entries=80)
    try:
        data = torch.arange(60 * 16, dtype=torch.int32).to(torch.uint8).cuda()
        assert cache.alloc(60, data) == 0
        gone = [7, 3, 4, 5, 59, 0, 41]
        cache.free_each(torch.tensor([[-1] + gone], dtype=torch.int32, device="cuda"))
        cache.free_each(torch.tensor([], dtype=torch.int32))
        stay = [a for a in range(60) if a not in gone]
        out, entry = cache.out_buffer(0, 60), torch.empty(len(stay), dtype=torch.int32, device="cuda")
        off = torch.empty(2, dtype=torch.int32, device="cuda")
        cache.step_group(0, torch.tensor(stay[:38], dtype=torch.int32, device="cuda").view(1, 1, -1), out, entry, off)
        cache.sync()
        assert torch.equal(out[0, :38], data.view(60, 16)[stay[:38]])
        for bad in (gone[0], 60):
            with pytest.raises(ula.UlaError):
                cache.free_each(torch.tensor([bad], dtype=torch.int32))
        assert cache.alloc(7, data[:7 * 16].clone()) == 60
        cache.sync()
    finally:
        cache.close()


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("R,Q,H,K", [(700, 1, 20, 100), (640, 1, 64, 128), (610, 1, 128, 40), (620, 2, 16, 5), (615, 2, 32, 77)])
def test_score_items_of_one_tile(R, Q, H, K, shared):
    """Four items of one tile or more in every block, for each number of columns: every repetition's bits are the first's."""
    from serving_step_sparse_gb300 import rows
    before, *case = score_case(R, Q, H, K, 500, R + K, pads=0.1, shared=shared)
    want = rows.score(before.clone(), *case, SCALE)
    check_score(want, score64(before, *case, SCALE))
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        differ += (rows.score(before.clone(), *case, SCALE) != want).sum()
    rows.sync()
    assert int(differ) == 0


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("R,Q,H,K", [(320, 2, 16, 60), (310, 2, 20, 100), (620, 1, 64, 40), (40, 4, 20, 700)])
def test_tree_repeats_its_bits(R, Q, H, K, shared):
    """Items of one tile, several in every block, and items that blocks share: every repetition's bits are the first's."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own, parent = tree_case(R, Q, H, K, 500, R + K, "random", shared, pads=0.1)
    want = rows.attend_tree(q, kv, entry, SCALE, own, parent)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(50):
        out, lse = rows.attend_tree(q, kv, entry, SCALE, own, parent)
        differ += (out != want[0]).sum() + (lse != want[1]).sum()
    rows.sync()
    assert int(differ) == 0


@pytest.mark.parametrize("R,Q,H,K", [(1, 1, 1, 300), (2, 3, 40, 500), (8, 3, 64, 2048)])
@pytest.mark.parametrize("below", [8.0, 20.0, 40.0])
def test_score_small_weights(R, Q, H, K, below):
    """Weights of e^-below of an attention's count as others do, beside those of a token whose weights are whole.
    Each is off by what the head of this file says, without a fixed point's share but for its last unit: a call of n
    weights, 4 at least, adds whole numbers of 2^-2e with e = 62 - ceil(log2 n), so a row's sum is off by half of one."""
    from serving_step_sparse_gb300 import rows
    before, q, kv, entry, address, lse = score_case(R, Q, H, K, K, R + K)
    lse += below
    entry[0, 0, : K // 2] = -1
    lse[0, 0] -= below
    first = address[0, 0].clone()
    address[0, 0] = torch.where(first % 2 == 0, first, -1)
    got = rows.score(torch.zeros_like(before), q, kv, entry, address, lse, SCALE).double().cpu().numpy()
    rows.sync()
    lat, rope = unpack(kv)
    keys, qd, zd = np.concatenate([lat, rope], axis=1), q.double().cpu().numpy(), lse.double().cpu().numpy()
    e, a = entry.cpu().numpy(), address.cpu().numpy()
    want, slack = np.zeros(len(got)), np.zeros(len(got))
    unit = 2.0 ** (-2 * (62 - max(2, math.ceil(math.log2(R * Q * H * K)))))
    for r in range(R):
        for i in range(Q):
            ok = (e[r, i] >= 0) & (a[r, i] >= 0)
            k, m = keys[e[r, i][ok]], zd[r, i][:, None]
            z, err = qd[r, i] @ k.T * SCALE, 2.0 ** -20 * SCALE * (np.abs(qd[r, i]) @ np.abs(k).T)
            p = np.exp(z - m)
            np.add.at(want, a[r, i][ok], p.sum(0))
            loss = p * (np.expm1(err + 2.0 ** -22 * (np.abs(z) + np.abs(m))) + 2.0 ** -21 + 2.0 ** -16)
            np.add.at(slack, a[r, i][ok], loss.sum(0) + unit / 2 * math.ceil(H / 128) + 2.0 ** -126 * H)
    assert (np.abs(got - want) <= slack + 2.0 ** -23 * want * 1.01).all()


def test_score_orders_what_is_hardly_seen():
    """Addresses whose weights are all small leave by them, not by age."""
    from serving_step_sparse_gb300 import rows
    n, heads = 64, 128
    _, kv, _, _ = attend_case(1, 1, 1, 1, n, 5)
    q = torch.zeros(16, 1, heads, 576, dtype=torch.bfloat16, device="cuda")
    order = torch.randperm(n, device="cuda").to(torch.int32)
    entry = order.expand(16, 1, n).contiguous()
    # logits of 0: a weight is e^-lse, and the later an address stands in the order the fewer tokens list it
    for i in range(16):
        entry[i, 0, n - 4 * i:] = -1
    lse = torch.full((16, 1, heads), 60.0, device="cuda")
    scores = rows.score(torch.zeros(n, device="cuda"), q, kv, entry, entry, lse, SCALE)
    assert (scores > 0).all()
    kept, dropped = rows.evict(scores, torch.arange(n, dtype=torch.int32, device="cuda")[None], torch.tensor([n], dtype=torch.int32, device="cuda"), n // 2)
    assert torch.equal(dropped[0], order[n // 2:].sort().values) and torch.equal(kept[0], order[:n // 2].sort().values)


RANGE = {"bf16": (5e17, 1e15, 1e-12, 1e-15), "f32": (5e17, 1e15, 1e-12, 1e-15), "f16": (6e4, 1e-4, 6e-8)}


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("width", [64, 128, 130, 576, 640, 1024])
def test_norm_range(width, dtype):
    """Heads at the ends of the range, and some channels there alone, beside heads of ordinary size.  (1,024 squares
    of 5e17 are 2.6e38; a square of 1e-15 / 2 is 2^-102, so its least bit of 24 is a normal number's.)"""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(width)
    rot, freq, axis = make_rotary(rng, 2, "halves")
    n, heads, at = 9, 8, width - 64
    pos = positions(rng, 2, n)
    pos_d = torch.from_numpy(pos).cuda()
    x = rng.uniform(0.5, 1, (n, heads, width)) * rng.choice([-1, 1], (n, heads, width))
    plain = torch.from_numpy(x).to(DT[dtype]).cuda()
    for i, size in enumerate(RANGE[dtype]):
        x[i, 1::2] *= size
        x[i + 4, 2, :3] *= size
    x = torch.from_numpy(x).to(DT[dtype]).cuda()
    w = torch.from_numpy(1 + 0.3 * rng.standard_normal(width)).float().cuda()
    for eps in (0.0, 1e-30, 1e-6):
        out = rows.norm_rotate(x, w, pos_d, rot, at=at, eps=eps)
        check_norm(out, x, w, eps, at, pos, freq, axis, "halves", dtype)
        assert torch.equal(out[:, 0], rows.norm_rotate(plain, w, pos_d, rot, at=at, eps=eps)[:, 0])
    if dtype != "f16":
        assert not rows.norm_rotate(torch.full_like(x, 1e20), w, pos_d, rot, at=at).any()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_pack_norm_range(dtype):
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(3)
    rot, freq, axis = make_rotary(rng, 2, "adjacent")
    n = 20
    x, k = rng.uniform(0.5, 1, (n, 512)), rng.uniform(0.5, 1, (n, 64))
    for i, size in enumerate(RANGE[dtype]):
        x[2 * i] *= size
        k[2 * i + 1] *= size
        x[2 * i + 1, 100:102] *= size
    latent, rope = torch.from_numpy(x).to(DT[dtype]).cuda(), torch.from_numpy(k).to(DT[dtype]).cuda()
    w, rw = torch.from_numpy(1 + 0.3 * rng.standard_normal(512)).float().cuda(), torch.from_numpy(1 + 0.3 * rng.standard_normal(64)).float().cuda()
    pos = positions(rng, 2, n)
    for eps in (0.0, 1e-30, 1e-6):
        got = rows.pack_norm(latent, rope, w, torch.from_numpy(pos).cuda(), rot, rope_weight=rw, eps=eps)
        check_pack_norm(got, latent, rope, w, rw, eps, pos, freq, axis, "adjacent")


def test_draft_tree_example_weights():
    """Every address's accumulated weights, as a part of them.  Heads and rows are normed (weights below 1.5, codes
    off by 2^-4), so |z| and sum |q k| * scale are at most 1.5^2 * 17 / 16 * 576 * 192^-0.5 < 100.  A logit is off by
    2^-20 * 100, and so is the lse, which has 2^-23 * 105 of its own and 2^-16 of its sum; the difference in units of
    log2 2^-22 * 205, the exponential 2^-21; 20 heads in fp32 are 20 * 2^-24, a score's 3 * 2 * 2 additions 12 * 2^-24:
    2.9e-4 in all."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_tree.py")
    spec = importlib.util.spec_from_file_location("draft_tree", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.run(steps=3, seed=1, check=True)[1] <= 2.9e-4
