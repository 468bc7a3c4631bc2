"""The operators on FP8 rows against plain implementations in 64 bits.

Tolerances, derived from the number formats:
  * an output rounded once to bf16 (f16, f32), which hold 8 (11, 24) significant bits, is off
    by at most half a unit of its last place, 2^-8 (2^-11, 2^-24) of its size, plus what the
    fp32 arithmetic before it loses;
  * rotary angles are exact to 2^-24 of a turn's half and sincospi to a few fp32 ulp:
    each turned pair is off by at most 2^-20 of its length before the rounding;
  * attention: logits are fp32 sums of 576 products, off by at most 2^-20 * sum |q k| *
    scale; probabilities enter the second product in 16 bits (relative 2^-8 at worst), so
    an output channel is off by at most 2^-8 * sum_e p_e |v_e| on top of its own rounding;
    logits off by d change a probability by a factor of at most e^(2d); and exp in fp32
    holds nothing below 2^-126 (its argument taken from a maximum that may lag by 2^8), so
    each row may lose 2^-118 * |v|.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
HALF_ULP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
SMALLEST = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24, "f32": 2.0 ** -149}


def _e4m3():
    v = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[b] = math.nan if (b & 127) == 127 else (-x if b & 128 else x)
    return v


E4M3 = _e4m3()


def unpack(rows: torch.Tensor):
    """rows uint8 [n][656] -> latent, rope in float64 numpy."""
    b = rows.cpu().numpy().reshape(-1, 656)
    codes = E4M3[b[:, :512]]
    scales = np.ascontiguousarray(b[:, 512:528]).view(np.float32).astype(np.float64)
    bits = np.ascontiguousarray(b[:, 528:]).view(np.uint16).astype(np.uint32) << 16
    return codes * np.repeat(scales, 128, axis=1), bits.view(np.float32).astype(np.float64)


def random_rows(n, rng, spread=0.3):
    """Rows of random codes (no NaN codes) and scales, as bytes."""
    codes = rng.integers(0, 256, (n, 512), dtype=np.uint8)
    codes[(codes & 127) == 127] = 0
    scales = (np.exp(spread * rng.standard_normal((n, 4))) / 200).astype(np.float32)
    rope = rng.standard_normal((n, 64)).astype(np.float32).view(np.uint32) >> 16
    return torch.from_numpy(np.concatenate(
        [codes, scales.view(np.uint8).reshape(n, 16),
         rope.astype(np.uint16).view(np.uint8).reshape(n, 128)], axis=1)).cuda()


# ------------------------------------------------------------------------------- rotary

def make_rotary(rng, axes, pairing):
    from serving_step_sparse_gb300 import rows
    freq = np.float32(10000.0) ** (-np.arange(32, dtype=np.float32) / 32)
    axis = rng.integers(0, axes, 32)
    axis[0], axis[31] = 0, axes - 1
    return rows.Rotary(freq.tolist(), axis.tolist(), pairing), freq.astype(np.float64), axis


def turned(x, pos, freq, axis, pairing, sign=1.0):
    x = np.asarray(x, dtype=np.float64)
    ang = pos.astype(np.float64)[axis].T * freq[None]            # [n][32]
    ang = ang.reshape(ang.shape[0], *([1] * (x.ndim - 2)), 32)
    c, s = np.cos(ang), sign * np.sin(ang)
    out = np.empty_like(x)
    ia, ib = ((slice(0, None, 2), slice(1, None, 2)) if pairing == "adjacent"
              else (slice(0, 32), slice(32, 64)))
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, a * s + b * c
    length = np.empty_like(x)
    length[..., ia] = length[..., ib] = np.hypot(a, b)
    return out, length


def positions(rng, axes, n, top=131072):
    pos = rng.integers(0, top, (axes, n)).astype(np.int32)
    pos[0, 0] = 0
    if n > 2:
        pos[0, 1], pos[axes - 1, 2] = 2 ** 30 + 12345, -7
    return pos


def check_turned(got, x, pos, freq, axis, pairing, dtype, sign=1.0):
    want, length = turned(x, pos, freq, axis, pairing, sign)
    tol = HALF_ULP[dtype] * np.abs(want) * 1.01 + 2.0 ** -20 * length + SMALLEST[dtype]
    assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,heads,axes", [(1, 1, 1), (3, 5, 3), (17, 64, 2), (700, 1, 4), (33, 128, 8)])
def test_rotate(n, heads, axes, dtype, pairing):
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(n * 131 + heads)
    rot, freq, axis = make_rotary(rng, axes, pairing)
    x = torch.from_numpy(rng.standard_normal((n, heads, 64))).to(DT[dtype]).cuda()
    pos = positions(rng, axes, n)
    pos_d = torch.from_numpy(pos).cuda()
    out = rows.rotate(x, pos_d, rot)
    check_turned(out, x.double().cpu(), pos, freq, axis, pairing, dtype)
    back = rows.rotate(x, pos_d, rot, inverse=True)
    check_turned(back, x.double().cpu(), pos, freq, axis, pairing, dtype, sign=-1.0)
    y = x.clone()
    assert rows.rotate(y, pos_d, rot, out=y) is y and torch.equal(y, out)  # in place


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset,head_stride,token_extra", [(0, 64, 0), (512, 576, 0), (8, 80, 16),
                                                            (1, 65, 3), (2, 66, 2), (512, 576, 1)])
def test_rotate_strides_and_alignment(dtype, offset, head_stride, token_extra):
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(offset + head_stride)
    n, heads = 37, 6
    for pairing in ("adjacent", "halves"):
        rot, freq, axis = make_rotary(rng, 3, pairing)
        store = torch.from_numpy(rng.standard_normal(
            offset + n * (heads * head_stride + token_extra) + 64)).to(DT[dtype]).cuda()
        view = store.as_strided((n, heads, 64), (heads * head_stride + token_extra, head_stride, 1), offset)
        x = view.clone()
        pos = positions(rng, 5, n)
        pos_d = torch.from_numpy(pos).cuda()
        dense = rows.rotate(view, pos_d, rot)            # strided in, dense out
        check_turned(dense, x.double().cpu(), pos, freq, axis, pairing, dtype)
        before = store.clone()
        rows.rotate(view, pos_d, rot, out=view)          # strided, in place
        assert torch.equal(view, dense)
        mask = torch.ones_like(store, dtype=torch.bool)
        mask.as_strided(view.shape, view.stride(), offset).fill_(False)
        assert torch.equal(store[mask], before[mask])    # nothing beside the channels
    assert torch.equal(rows.rotate(x[:, 0], pos_d, rot), dense[:, 0])  # no head axis


def test_rotate_gradient():
    """The inverse turn is the gradient: <g, rotate(x)> = <rotate_inverse(g), x>, and it agrees
    with central differences of the turn (linear in x, so exact up to fp32 rounding: each inner
    product of 64 terms is off by at most 2^-18 of the vectors' lengths)."""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(3)
    rot, freq, axis = make_rotary(rng, 3, "halves")
    pos = torch.from_numpy(positions(rng, 3, 9)).cuda()
    x = torch.from_numpy(rng.standard_normal((9, 2, 64))).float().cuda()
    g = torch.from_numpy(rng.standard_normal((9, 2, 64))).float().cuda()
    grad = rows.rotate(g, pos, rot, inverse=True).double()
    size = (x.norm() * g.norm()).double()
    assert abs((g.double() * rows.rotate(x, pos, rot).double()).sum() - (grad * x.double()).sum()) <= 2.0 ** -18 * size
    for _ in range(8):
        d = torch.from_numpy(rng.standard_normal((9, 2, 64))).float().cuda()
        step = (rows.rotate(x + d, pos, rot).double() - rows.rotate(x - d, pos, rot).double()) / 2
        assert abs((g.double() * step).sum() - (grad * d.double()).sum()) <= 2.0 ** -18 * (
            g.norm() * (x.norm() + d.norm())).double()


# ------------------------------------------------------------------------------- pack

@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,layers", [(1, 1), (7, 4), (8, 1), (129, 3), (1000, 1)])
def test_pack(n, layers, dtype, pairing):
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(n * 7 + layers)
    rot, freq, axis = make_rotary(rng, 3, pairing)
    x = rng.standard_normal((n, 512)) * np.exp(rng.standard_normal((n, 1)))
    x[0, :128] = 0                      # a block of zeros
    x[n // 2, 128:256] *= 1e-4          # blocks of other sizes
    x[n - 1, 384:] *= 50
    latent = torch.from_numpy(x).to(DT[dtype]).cuda()
    rope = torch.from_numpy(rng.standard_normal((n, 64))).to(DT[dtype]).cuda()
    pos = positions(rng, 3, n)
    dest = torch.full((n, layers, 656), 0xA5, dtype=torch.uint8, device="cuda")
    got = rows.pack(latent, rope, torch.from_numpy(pos).cuda(), rot, dest[:, layers - 1])
    assert got.data_ptr() == dest[:, layers - 1].data_ptr()
    assert (dest[:, :layers - 1] == 0xA5).all()
    b = got.cpu().numpy()
    v = latent.double().cpu().numpy().reshape(n, 4, 128)
    scale = np.ascontiguousarray(b[:, 512:528]).view(np.float32).astype(np.float64)
    want = np.maximum(np.abs(v).max(-1) / 448, 2.0 ** -126)
    assert (np.abs(scale - want) <= 2.0 ** -23 * want).all()
    codes = E4M3[b[:, :512]].reshape(n, 4, 128)
    y = v / scale[..., None]
    # the nearest e4m3 value: half the spacing around |y|, and the quotient's fp32 roundings
    spacing = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    assert (np.abs(codes - y) <= spacing / 2 + 2.0 ** -21 * np.abs(y)).all()
    got_rope = torch.from_numpy(np.ascontiguousarray(b[:, 528:])).view(torch.bfloat16)
    check_turned(got_rope, rope.double().cpu(), pos, freq, axis, pairing, "bf16")


def test_pack_not_finite():
    """A block with a NaN or an infinity stands for NaN throughout; its neighbours are whole."""
    from serving_step_sparse_gb300 import rows
    rot = rows.Rotary([0.0] * 32)
    latent = torch.ones(3, 512, device="cuda")
    latent[0, 5], latent[1, 200], latent[2, 511] = math.nan, math.inf, -math.inf
    got = rows.pack(latent, torch.zeros(3, 64, device="cuda"),
                    torch.zeros(3, dtype=torch.int32, device="cuda"), rot)
    lat, rope = unpack(got)
    for t, blk in ((0, 0), (1, 1), (2, 3)):
        v = lat[t].reshape(4, 128)
        assert np.isnan(v[blk]).all()
        rest = [b for b in range(4) if b != blk]
        assert (np.abs(v[rest] - 1) <= 2.0 ** -20).all()   # 1 is the block's largest: code 448
    assert (rope == 0).all()


def test_pack_quotients():
    """Codes are those of the fp32 quotient x / scale, correctly rounded, for values at and next
    to the middle of two codes (a quotient one unit off would cross it)."""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(11)
    mids = (E4M3[1:126] + E4M3[2:127]) / 2
    n = 400
    top = np.exp(3 * rng.standard_normal((n, 4, 1))).astype(np.float32)
    scale = np.maximum(top / np.float32(448), np.float32(2.0 ** -126))
    x = (rng.choice(mids, (n, 4, 128)) * rng.choice([-1, 1], (n, 4, 128)) * scale).astype(np.float32)
    x = x.view(np.int32) + rng.integers(-2, 3, x.shape).astype(np.int32)
    x = np.clip(x.view(np.float32), -top, top)
    x[:, :, 0] = top[:, :, 0]
    latent = torch.from_numpy(x.reshape(n, 512)).cuda()
    got = rows.pack(latent, torch.zeros(n, 64, device="cuda"),
                    torch.zeros(n, dtype=torch.int32, device="cuda"), rows.Rotary([0.0] * 32))
    want = torch.from_numpy((x / scale).reshape(n, 512)).to(torch.float8_e4m3fn)
    assert torch.equal(got[:, :512].cpu(), want.view(torch.uint8))


def test_pack_strides():
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(5)
    rot, _, _ = make_rotary(rng, 2, "adjacent")
    n = 21
    for dtype in DT.values():
        wide = torch.from_numpy(rng.standard_normal((n, 600))).to(dtype).cuda()
        pos = torch.from_numpy(positions(rng, 2, n)).cuda()
        for at in (0, 1, 8, 13):                      # an unaligned start, rows apart
            latent, rope = wide[:, at:at + 512], wide[:, at + 513:at + 577]
            want = rows.pack(latent.contiguous(), rope.contiguous(), pos, rot)
            assert torch.equal(rows.pack(latent, rope, pos, rot), want)
        turned_over = torch.flip(wide, [1]).t().contiguous().t()   # channels apart
        assert torch.equal(rows.pack(turned_over[:, :512], turned_over[:, 512:576], pos, rot),
                           rows.pack(turned_over[:, :512].contiguous(),
                                     turned_over[:, 512:576].contiguous(), pos, rot))


# ------------------------------------------------------------------------------- attend

def attend64(q, rows, entry, scale, own=None):
    """(out, lse, slack): slack bounds an output channel's error per unit (see the top)."""
    R, Q, H, _ = q.shape
    lat_all, rope_all = unpack(rows) if rows.shape[0] else (np.zeros((0, 512)), np.zeros((0, 64)))
    qd = q.double().cpu().numpy()
    e = entry.cpu().numpy()
    out, lse = np.zeros((R, Q, H, 512)), np.full((R, Q, H), -np.inf)
    slack, zslack = np.zeros((R, Q, H, 512)), np.zeros((R, Q, H))
    for r in range(R):
        for i in range(Q):
            idx = e[r, i][(e[r, i] >= 0) & (e[r, i] < rows.shape[0])]
            lat, rope = lat_all[idx], rope_all[idx]
            if own is not None:
                ol, orp = unpack(own[r, :i + 1].contiguous())
                lat, rope = np.concatenate([lat, ol]), np.concatenate([rope, orp])
            if not len(lat):
                continue
            keys = np.concatenate([lat, rope], axis=1)
            z = qd[r, i] @ keys.T * scale
            zslack[r, i] = (2.0 ** -20 * abs(scale) * (np.abs(qd[r, i]) @ np.abs(keys).T)).max(-1)
            top = z.max(-1, keepdims=True)
            p = np.exp(z - top)
            lse[r, i] = (top + np.log(p.sum(-1, keepdims=True)))[:, 0]
            p /= p.sum(-1, keepdims=True)
            out[r, i] = p @ lat
            slack[r, i] = p @ np.abs(lat) + 2.0 ** -110 * np.abs(lat).sum(0)
    return out, lse, slack, zslack


def check_attend(got, want):
    (o, z), (out, lse, slack, zslack) = got, want
    o, z = o.double().cpu().numpy(), z.double().cpu().numpy()
    none = np.isneginf(lse)
    assert np.array_equal(np.isneginf(z), none)
    assert (o[none] == 0).all()
    ok = ~none
    # lse: the largest logit's error, and exp, log and the sum in fp32
    assert (np.abs(z - lse)[ok] <= (zslack + 2.0 ** -20 * (1 + np.abs(lse)))[ok]).all()
    tol = 2.0 ** -8 * np.abs(out) * 1.01 + (2.0 ** -8 + np.expm1(2 * zslack[..., None])) * slack + 2.0 ** -133
    assert (np.abs(o - out) <= tol)[ok].all()


def attend_case(R, Q, H, K, n_rows, seed, pads=0.0, own=False, qscale=1.0, spread=0.3):
    rng = np.random.default_rng(seed)
    q = torch.from_numpy(qscale * rng.standard_normal((R, Q, H, 576))).to(torch.bfloat16).cuda()
    rows = random_rows(n_rows, rng, spread)
    entry = rng.integers(0, max(n_rows, 1), (R, Q, K)).astype(np.int32)
    if pads:
        entry[rng.random(entry.shape) < pads] = -1
    own_rows = random_rows(R * Q, rng, spread).view(R, Q, 656) if own else None
    return q, rows, torch.from_numpy(entry).cuda(), own_rows


SCALE = 192 ** -0.5


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("R,Q,H,K", [
    (1, 1, 1, 1), (1, 1, 16, 127), (1, 1, 17, 128), (2, 3, 32, 129), (1, 2, 33, 255),
    (3, 1, 64, 256), (1, 1, 65, 300), (2, 2, 128, 517), (1, 1, 130, 64), (1, 4, 20, 2048),
    (40, 1, 8, 96), (1, 1, 64, 8192)])
def test_attend(R, Q, H, K, own):
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own_rows = attend_case(R, Q, H, K, max(1, 3 * K // 2), R * 1000 + H + K, own=own)
    got = rows.attend(q, kv, entry, SCALE, own_rows=own_rows)
    check_attend(got, attend64(q, kv, entry, SCALE, own_rows))
    rows.sync()


@pytest.mark.parametrize("H", [5, 64, 100])
@pytest.mark.parametrize("own", [False, True])
def test_attend_pads(H, own):
    """Pads anywhere, whole tiles of pads, a query without rows, entries out of range."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own_rows = attend_case(3, 2, H, 700, 500, H, pads=0.3, own=own)
    entry[0, 0] = -1
    entry[0, 1, :400] = -1
    entry[1, 0, 130:] = -1
    entry[1, 1, ::2] = torch.iinfo(torch.int32).min
    entry[2, 0, 1::3] = 500
    entry[2, 1, 5] = torch.iinfo(torch.int32).max
    got = rows.attend(q, kv, entry, SCALE, own_rows=own_rows)
    check_attend(got, attend64(q, kv, entry, SCALE, own_rows))


def test_attend_empty_lengths():
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own_rows = attend_case(2, 3, 24, 0, 4, 1, own=True)
    check_attend(rows.attend(q, kv, entry, SCALE), attend64(q, kv, entry, SCALE))
    check_attend(rows.attend(q, kv, entry, SCALE, own_rows=own_rows),
                 attend64(q, kv, entry, SCALE, own_rows))
    entry = torch.zeros(2, 3, 5, dtype=torch.int32, device="cuda")
    none = kv[:0].contiguous()
    check_attend(rows.attend(q, none, entry, SCALE), attend64(q, none, entry, SCALE))
    out, lse = rows.attend(q[:0], kv, entry[:0], SCALE)
    assert out.shape == (0, 3, 24, 512) and lse.shape == (0, 3, 24)
    out, lse = rows.attend(q[:, :, :0], kv, entry, SCALE)
    assert out.shape == (2, 3, 0, 512)


@pytest.mark.parametrize("qscale,spread", [(30.0, 0.3), (1e-3, 0.3), (1.0, 4.0), (8.0, 2.0)])
def test_attend_sizes_of_values(qscale, spread):
    """Peaked and flat distributions, scales over many orders: running maxima that move."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own_rows = attend_case(2, 2, 40, 900, 900, 77, own=True, qscale=qscale, spread=spread)
    got = rows.attend(q, kv, entry, SCALE, own_rows=own_rows)
    check_attend(got, attend64(q, kv, entry, SCALE, own_rows))


def test_attend_growing_logits():
    """Rows ordered by their logit, ascending and descending: the maximum moves in every tile,
    or is the first one; and a negative scale."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, _ = attend_case(1, 1, 48, 1500, 1500, 5, qscale=20.0)
    q[:] = q[:, :, :1]
    lat, rope = unpack(kv)
    z = np.concatenate([lat, rope], 1) @ q[0, 0, 0].double().cpu().numpy()
    for order in (np.argsort(z), np.argsort(-z)):
        entry[0, 0] = torch.from_numpy(order.astype(np.int32)).cuda()
        for scale in (SCALE, -SCALE):
            check_attend(rows.attend(q, kv, entry, scale), attend64(q, kv, entry, scale))


def test_attend_block_sizes_differ():
    """Blocks of channels, tokens and heads of very different sizes keep their own precision."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, _ = attend_case(1, 2, 64, 400, 400, 9)
    sc = kv[:, 512:528].contiguous().view(torch.float32)
    sc[:, 1] *= 2.0 ** -40
    sc[:, 2] *= 2.0 ** 20
    sc[:200, 3] *= 2.0 ** -60
    sc[300:] *= 2.0 ** 10
    kv[:, 512:528] = sc.view(torch.uint8)
    q[:, :, ::3] *= 2.0 ** -50
    q[:, :, 1::3] *= 2.0 ** -20
    q[:, :, :, 256:384] *= 2.0 ** -30     # block 2's share of the logits
    check_attend(rows.attend(q, kv, entry, SCALE), attend64(q, kv, entry, SCALE))


def test_attend_not_finite():
    """A NaN row poisons the queries that select it and no others; in rows that a query does
    not select, NaN and infinity count for nothing; so does a NaN head for other heads."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, _ = attend_case(1, 3, 33, 260, 300, 21)
    bad = kv.clone()
    bad[299, 512:528] = torch.tensor([math.nan] * 4).view(torch.uint8).cuda()
    bad[298, :512] = 0x7F                                       # NaN codes under whole scales
    bad[297, 528:] = 0xFF                                       # NaN rope
    entry = entry.clamp_max(296)
    clean = rows.attend(q, kv, entry, SCALE)
    same = rows.attend(q, bad, entry, SCALE)
    assert torch.equal(clean[0], same[0]) and torch.equal(clean[1], same[1])
    entry[0, 1, 77] = -1
    entry[0, 0, 3], entry[0, 2, 200] = 299, 298
    out, lse = rows.attend(q, bad, entry, SCALE)
    assert torch.isnan(out[0, 0]).all() and torch.isnan(lse[0, 0]).all()
    assert torch.isnan(out[0, 2]).all() and torch.isnan(lse[0, 2]).all()
    want = attend64(q[:, 1:2], kv, entry[:, 1:2], SCALE)
    check_attend((out[:, 1:2], lse[:, 1:2]), want)
    entry[0, 0, 3], entry[0, 2, 200] = 0, 297
    out, lse = rows.attend(q, bad, entry, SCALE)
    assert torch.isnan(out[0, 2]).all() and not torch.isnan(out[0, :2]).any()
    q2 = q.clone()
    q2[0, 0, 7, 100] = math.nan
    q2[0, 0, 8, 570] = math.inf
    o1, l1 = rows.attend(q2, kv, entry.clamp_max(296), SCALE)
    o0, l0 = rows.attend(q, kv, entry.clamp_max(296), SCALE)
    others = [h for h in range(33) if h not in (7, 8)]
    assert torch.equal(o1[0, 0, others], o0[0, 0, others]) and torch.equal(l1[0, 0, others], l0[0, 0, others])
    assert torch.isnan(o1[0, 0, 7]).all() and torch.isnan(l1[0, 0, 7])
    assert torch.isnan(o1[0, 0, 8]).all()


def test_attend_strides():
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own_rows = attend_case(3, 2, 12, 200, 150, 4, own=True)
    want = rows.attend(q, kv, entry, SCALE, own_rows=own_rows)
    wide = torch.zeros(3, 2, 12, 640, dtype=torch.bfloat16, device="cuda")
    wide[..., 8:584] = q
    heads_first = q.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    odd = torch.zeros(3, 2, 12, 577, dtype=torch.bfloat16, device="cuda")
    odd[..., 1:] = q
    own_wide = torch.zeros(3, 4, 2, 656, dtype=torch.uint8, device="cuda")
    own_wide[:, 1:3, 1] = own_rows
    back = torch.zeros(200, 2, 3, dtype=torch.int32, device="cuda")
    back[:] = entry.permute(2, 1, 0)
    for qq in (wide[..., 8:584], heads_first, odd[..., 1:]):
        got = rows.attend(qq, kv, back.permute(2, 1, 0), SCALE, own_rows=own_wide[:, 1:3, 1])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    got = rows.attend(q, kv, entry, SCALE, own_rows=own_rows, out=out, lse=lse)
    assert got[0] is out and got[1] is lse and torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("R,Q,H,K,own", [
    (12, 1, 16, 1024, False), (5, 2, 20, 777, True), (16, 1, 32, 600, False), (38, 2, 64, 129, True),
    (20, 1, 40, 512, False), (37, 1, 64, 300, False), (9, 4, 130, 200, False), (38, 1, 1, 380, True)])
def test_attend_few_tiles(R, Q, H, K, own):
    """Numbers of tiles about as large as the GPU: items of two to eight tiles in as many blocks.
    Parts without rows, a query token without rows, one with a single row in its last tile."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own_rows = attend_case(R, Q, H, K, 500, R + K, pads=0.1, own=own)
    entry[0, 0, :] = -1
    entry[1, 0, :128] = -1
    entry[2, 0, 128:] = -1
    entry[3, -1, :K - 1] = -1
    got = rows.attend(q, kv, entry, SCALE, own_rows=own_rows)
    check_attend(got, attend64(q, kv, entry, SCALE, own_rows))
    bad = kv.clone()
    bad[499, 512:528] = torch.tensor([math.nan] * 4).view(torch.uint8).cuda()
    entry = torch.where(entry == 499, 498, entry)
    clean = rows.attend(q, bad, entry, SCALE, own_rows=own_rows)
    entry[4, 0, K - 1] = 499
    out, lse = rows.attend(q, bad, entry, SCALE, own_rows=own_rows)
    assert torch.isnan(out[4, 0]).all() and torch.isnan(lse[4, 0]).all()
    out[4, 0], lse[4, 0] = clean[0][4, 0], clean[1][4, 0]
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
    rows.sync()


def test_attend_far_rows():
    """A gathered buffer past 2^32 bytes."""
    from serving_step_sparse_gb300 import rows
    n = 2 ** 32 // 656 + 1000
    big = torch.zeros(n, 656, dtype=torch.uint8, device="cuda")
    q, kv, entry, _ = attend_case(1, 1, 16, 300, 300, 6)
    big[-300:] = kv
    want = rows.attend(q, kv, entry, SCALE)
    got = rows.attend(q, big, entry + (n - 300), SCALE)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attend_repeats():
    """The same call gives the same bits."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own_rows = attend_case(4, 3, 64, 1000, 900, 8, own=True)
    a = rows.attend(q, kv, entry, SCALE, own_rows=own_rows)
    for _ in range(5):
        b = rows.attend(q, kv, entry, SCALE, own_rows=own_rows)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("R,Q,H,K", [(220, 1, 64, 11), (55, 2, 69, 11), (400, 1, 3, 100), (90, 2, 20, 300)])
def test_attend_many_items(R, Q, H, K):
    """More query tokens than blocks, so that a block takes several whole items, many times
    over: blocks' warps drift apart and must not meet another tile's addresses."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own_rows = attend_case(R, Q, H, K, 500, R + K, pads=0.2, own=True)
    want = rows.attend(q, kv, entry, SCALE, own_rows=own_rows)
    check_attend(want, attend64(q, kv, entry, SCALE, own_rows))
    for _ in range(300):
        got = rows.attend(q, kv, entry, SCALE, own_rows=own_rows)
    rows.sync()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("R,Q,H,K", [
    (161, 1, 64, 700), (200, 1, 24, 1100), (153, 1, 16, 2000), (155, 2, 8, 260), (77, 2, 128, 150)])
def test_attend_whole_and_shared_items(R, Q, H, K):
    """Somewhat more query tokens (times 64 heads) than blocks: some are worked on whole, the rest
    by several blocks each, fewer than there are, or all."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, _ = attend_case(R, Q, H, K, 700, R + K, pads=0.05)
    got = rows.attend(q, kv, entry, SCALE)
    check_attend(got, attend64(q, kv, entry, SCALE))
    for _ in range(20):
        again = rows.attend(q, kv, entry, SCALE)
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    rows.sync()


def test_attend_other_stream():
    """Calls on streams of their own: inputs and temporaries are held until they have run."""
    from serving_step_sparse_gb300 import rows
    streams = [torch.cuda.Stream() for _ in range(3)]
    cases = [attend_case(2, 2, 40, 600, 500, 30 + s) for s in range(3)]
    want = [rows.attend(q, kv, e, SCALE) for q, kv, e, _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s, (q, kv, e, _) in zip(streams, cases):
            odd = torch.zeros(*q.shape[:3], 577, dtype=torch.bfloat16, device="cuda")
            odd[..., 1:] = q
            s.wait_stream(torch.cuda.current_stream())
            got.append(rows.attend(odd[..., 1:], kv, e, SCALE, stream=s))
            del odd
            torch.zeros(2, 2, 40, 577, dtype=torch.bfloat16, device="cuda").fill_(7.0)
    torch.cuda.synchronize()
    for i, (o, z) in enumerate(got):
        assert torch.equal(o, want[i % 3][0]) and torch.equal(z, want[i % 3][1])


# ------------------------------------------------------------------------------- join

def join64(outs, lses):
    z = np.stack([x.double().cpu().numpy() for x in lses])
    o = np.stack([x.double().cpu().numpy() for x in outs])
    top = z.max(0)
    ref = np.where(np.isneginf(top), 0.0, top)
    w = np.exp(z - ref)
    total = w.sum(0)
    p = w / np.where(total == 0, 1, total)
    o = np.where(np.isneginf(z)[..., None], 0, o)
    with np.errstate(divide="ignore"):
        lse = ref + np.log(total)
    return (o * p[..., None]).sum(0), lse, (np.abs(o) * p[..., None]).sum(0)


@pytest.mark.parametrize("parts", [1, 2, 3, 8])
@pytest.mark.parametrize("shape", [(1,), (3,), (5, 7), (2, 3, 64)])
def test_join(parts, shape):
    """fp32 arithmetic (each weight and sum off by at most 2^-20), rounded once to bf16."""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(parts)
    outs = [torch.from_numpy(rng.standard_normal((*shape, 512))).to(torch.bfloat16).cuda() for _ in range(parts)]
    lses = [torch.from_numpy(5 * rng.standard_normal(shape)).float().cuda() for _ in range(parts)]
    for p in range(parts):
        lses[p].view(-1)[p % lses[p].numel()] = -math.inf
        lses[p].view(-1)[-1] = -math.inf
        outs[p].view(-1, 512)[-1] = math.nan                    # (not read where lse is -inf)
    want, lse, slack = join64(outs, lses)
    o, z = rows.join(outs, lses)
    o, z = o.double().cpu().numpy(), z.double().cpu().numpy()
    none = np.isneginf(lse)
    assert np.array_equal(np.isneginf(z), none) and (o[none] == 0).all()
    assert (np.abs(z - lse)[~none] <= 2.0 ** -20 * (1 + np.abs(lse[~none]))).all()
    assert (np.abs(o - want) <= 2.0 ** -8 * 1.01 * np.abs(want) + 2.0 ** -18 * slack + 2.0 ** -133).all()
    keep = [x.clone() for x in outs], [x.clone() for x in lses]
    again = rows.join(outs, lses, out=outs[0], lse=lses[0])     # in place of the first part
    assert again[0] is outs[0]
    first = rows.join(*keep)
    assert torch.equal(first[0], outs[0]) and torch.equal(first[1], lses[0])


def test_join_of_attends():
    """Two halves of a selection, joined, against the whole one (TP: local and remote rows)."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, _ = attend_case(3, 2, 24, 500, 400, 12, pads=0.05)
    odd = (entry & 1).bool()
    a = rows.attend(q, kv, torch.where(odd, entry, -1), SCALE)
    b = rows.attend(q, kv, torch.where(odd, -1, entry), SCALE)
    o, z = rows.join([a[0], b[0]], [a[1], b[1]])
    out, lse, slack, zslack = attend64(q, kv, entry, SCALE)
    assert (np.abs(z.double().cpu().numpy() - lse) <= zslack + 2.0 ** -19 * (1 + np.abs(lse))).all()
    # each half was rounded to bf16 as well
    tol = 2.0 ** -8 * 1.01 * np.abs(out) + (2.0 ** -8 + 2.0 ** -8 + np.expm1(2 * zslack[..., None])) * slack
    assert (np.abs(o.double().cpu().numpy() - out) <= tol).all()


# ------------------------------------------------------------------------------- refusals

def test_refusals():
    from serving_step_sparse_gb300 import rows, ula
    q, kv, entry, own_rows = attend_case(2, 2, 8, 16, 16, 1, own=True)
    pos = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    rot = rows.Rotary([1.0] * 32)
    x = torch.zeros(4, 8, 64, device="cuda")
    bad = [
        lambda: rows.Rotary([1.0] * 31),
        lambda: rows.Rotary([1.0] * 32, [8] * 32),
        lambda: rows.Rotary([1.0] * 32, pairing="thirds"),
        lambda: rows.rotate(x[..., :32], pos, rot),
        lambda: rows.rotate(x.double(), pos, rot),
        lambda: rows.rotate(x, pos.long(), rot),
        lambda: rows.rotate(x, pos[:, :3], rot),
        lambda: rows.rotate(x, pos, rows.Rotary([1.0] * 32, [0] * 31 + [1])),
        lambda: rows.rotate(x, pos, rot, out=x.half()),
        lambda: rows.rotate(x, pos.cpu(), rot),
        lambda: rows.rotate(x.cpu(), pos.cpu(), rot),
        lambda: rows.pack(x[:, 0], x[:, 0], pos, rot),
        lambda: rows.pack(torch.zeros(4, 512, device="cuda"), x[:, 0].half(), pos, rot),
        lambda: rows.pack(torch.zeros(4, 512, device="cuda"), x[:, 0], pos, rot,
                          torch.zeros(4, 640, dtype=torch.uint8, device="cuda")),
        lambda: rows.pack(torch.zeros(4, 512, device="cuda"), x[:, 0], pos, rot,
                          torch.zeros(1, 656, dtype=torch.uint8, device="cuda").expand(4, 656)),
        lambda: rows.attend(q.float(), kv, entry, SCALE),
        lambda: rows.attend(q[..., :512], kv, entry, SCALE),
        lambda: rows.attend(q, kv[:, :640], entry, SCALE),
        lambda: rows.attend(q, kv[::2], entry, SCALE),
        lambda: rows.attend(q, kv, entry.long(), SCALE),
        lambda: rows.attend(q, kv, entry[:1], SCALE),
        lambda: rows.attend(q, kv, entry, SCALE, own_rows=own_rows[:1]),
        lambda: rows.attend(q, kv, entry, SCALE, out=torch.empty(2, 2, 8, 512, device="cuda")),
        lambda: rows.attend(q, kv.cpu(), entry, SCALE),
        lambda: rows.join([], []),
        lambda: rows.join([q[..., :512]], [entry[..., :8].float()]),
        lambda: rows.join([torch.zeros(3, 512, dtype=torch.bfloat16, device="cuda")] * 9,
                          [torch.zeros(3, device="cuda")] * 9),
        lambda: rows.join([torch.zeros(3, 512, dtype=torch.bfloat16, device="cuda")],
                          [torch.zeros(4, device="cuda")]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {i} was accepted")
    lat = torch.zeros(4, 512, device="cuda")
    store = torch.zeros(4 * 656 + 64, dtype=torch.uint8, device="cuda")
    with pytest.raises(ula.UlaError) as e:                       # rows that are not 16-byte aligned
        rows.pack(lat, x[:, 0], pos, rot, store[8:8 + 4 * 656].view(4, 656))
    assert e.value.code == ula.ERR_INVALID_ARG
    with pytest.raises(ula.UlaError):
        rows.pack(lat, x[:, 0], pos, rot, store.as_strided((4, 656), (664, 1)))
    with pytest.raises(ula.UlaError):
        rows.rotate(x, pos, rows.Rotary([math.inf] + [1.0] * 31))
    with pytest.raises(ula.UlaError):
        rows.attend(q, store[8:8 + 3 * 656].view(3, 656), entry, SCALE)
    rows.sync()


# ------------------------------------------------------------------------------- together

def test_decode_layers_example():
    """The operators with the cache, as a decode step uses them, against a dense computation in
    64 bits.  Outputs are averages of latents of unit size (at most 6): rounded to bf16 once
    for each of two parts and once for the joined result (2^-8 each), with the probabilities'
    2^-8: off by at most 4 * 2^-8 * 6."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_layers.py")
    spec = importlib.util.spec_from_file_location("decode_layers", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.run(steps=2, seed=1, check=True) <= 4 * 2.0 ** -8 * 6


def test_attend_partitions_of_tp():
    """TP mode: a rank's local and remote rows, two buffers with entry rows of their own, attended
    to separately and joined, against one buffer with all of them."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, _ = attend_case(4, 2, 24, 300, 600, 55, pads=0.05)
    remote = (torch.arange(600, device="cuda") % 2).bool()
    index = torch.cumsum(remote, 0).to(torch.int32) - 1
    other = torch.cumsum(~remote, 0).to(torch.int32) - 1
    at = entry.clamp_min(0).long()
    here = torch.where((entry >= 0) & ~remote[at], other[at], -1)
    there = torch.where((entry >= 0) & remote[at], index[at], -1)
    a = rows.attend(q, kv[~remote].contiguous(), here, SCALE)
    b = rows.attend(q, kv[remote].contiguous(), there, SCALE)
    o, z = rows.join([a[0], b[0]], [a[1], b[1]])
    out, lse, slack, zslack = attend64(q, kv, entry, SCALE)
    assert (np.abs(z.double().cpu().numpy() - lse) <= zslack + 2.0 ** -19 * (1 + np.abs(lse))).all()
    tol = 2.0 ** -8 * 1.01 * np.abs(out) + (2.0 ** -8 + 2.0 ** -8 + np.expm1(2 * zslack[..., None])) * slack
    assert (np.abs(o.double().cpu().numpy() - out) <= tol).all()


def test_rotary_copies():
    """A rotary that was copied or pickled turns by its own frequencies."""
    import copy
    import pickle
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(61)
    x = torch.from_numpy(rng.standard_normal((9, 4, 64))).float().cuda()
    pos = torch.from_numpy(positions(rng, 3, 9)).cuda()
    rot, _, _ = make_rotary(rng, 3, "halves")
    want = rows.rotate(x, pos, rot)
    others = [copy.deepcopy(rot), pickle.loads(pickle.dumps(rot))]
    rot.config.freq[:] = [0.0] * 32
    for other in others:
        assert torch.equal(rows.rotate(x, pos, other), want)


@pytest.mark.parametrize("R,H,K", [
    (1, 16, 100), (1, 20, 600), (2, 64, 2048), (160, 64, 300), (300, 8, 64),
    (12, 16, 1024), (16, 32, 600), (20, 40, 512)])        # (the last three: clusters)
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_attend_empty_query_not_finite(R, H, K, bad):
    """A query token that selects nothing gets 0 and -inf whatever its query holds, an unused
    query slot of a batch for instance; the others keep their bits."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, _ = attend_case(R, 1, H, K, 300, R + H + K, pads=0.1)
    empty = sorted({0, R - 1})
    entry[empty] = -1
    entry[empty, 0, K // 2:] = 300                         # out of range selects nothing either
    want = rows.attend(q, kv, entry, SCALE)
    q[empty[0]] = bad
    q[empty[-1], 0, :, ::97] = bad
    for e in (entry, entry[:, :, :0]):
        out, lse = rows.attend(q, kv, e, SCALE)
        assert (out[empty] == 0).all() and torch.isneginf(lse[empty]).all()
    out, lse = rows.attend(q, kv, entry, SCALE)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    rows.sync()


def test_attend_row_not_there_not_finite():
    """One row among pads: a query of NaN or infinity is that row's answer, not the pads'."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own_rows = attend_case(2, 3, 24, 300, 50, 3, own=True)
    kv[7, :128] = 0x38                                     # codes of 1 in the block in question
    kv[7, 512:516] = torch.tensor([1.0]).view(torch.uint8).cuda()
    entry[:] = -1
    entry[0, 0, 131] = 7
    q[0, 0, 5, :128] = -math.inf                           # that row's logit: -inf
    q[0, 0, 6, 3] = math.inf
    q[0, 0, 7, 3] = math.nan
    out, lse = rows.attend(q, kv, entry, SCALE)
    assert torch.isneginf(lse[0, 0, 5]) and (out[0, 0, 5] == 0).all()
    assert torch.isnan(out[0, 0, 6]).all() and torch.isnan(out[0, 0, 7]).all()
    rest = [h for h in range(24) if h not in (5, 6, 7)]
    check_attend((out[:, :, rest], lse[:, :, rest]), attend64(q[:, :, rest], kv, entry, SCALE))


def gives_up(case, barrier):
    """A call in which one barrier never opens: it ends, its error is reported once, and the next
    call is whole."""
    from serving_step_sparse_gb300 import rows, ula
    q, kv, entry, own_rows = case
    want = rows.attend(q, kv, entry, SCALE, own_rows=own_rows)
    rows.sync()
    ula.ula_rows_debug_hold(barrier)
    try:
        rows.attend(q, kv, entry, SCALE, own_rows=own_rows)
    finally:
        ula.ula_rows_debug_hold(-1)
    with pytest.raises(ula.UlaError) as e:
        rows.sync()
    assert e.value.code == ula.ERR_TIMEOUT
    rows.sync()
    got = rows.attend(q, kv, entry, SCALE, own_rows=own_rows)
    rows.sync()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("barrier", range(23))
def test_attend_gives_up(barrier):
    """Every barrier, with several tiles in a block and items that blocks share."""
    gives_up(attend_case(90, 2, 20, 300, 500, barrier, own=True), barrier)


@pytest.mark.parametrize("R,Q,H,K", [
    (1, 1, 64, 100), (12, 1, 16, 1024), (37, 1, 64, 300)])      # (the last two: clusters)
@pytest.mark.parametrize("barrier", [4, 5, 17, 19, 21])
def test_attend_gives_up_elsewhere(R, Q, H, K, barrier):
    """Single tiles, and clusters, whose blocks all have to meet."""
    gives_up(attend_case(R, Q, H, K, 500, R + H, pads=0.1), barrier)


def test_sync_of_several_streams():
    """A wait that ran out on one stream is reported by every stream's next sync, once by each."""
    from serving_step_sparse_gb300 import rows, ula
    q, kv, entry, _ = attend_case(1, 1, 16, 64, 64, 1)
    streams = [torch.cuda.Stream() for _ in range(3)] + [torch.cuda.current_stream()]
    for s in streams:
        try:
            rows.sync(s)
        except ula.UlaError:
            pass                                            # (an earlier test's)
    for failing in (1, 3):
        ula.ula_rows_debug_hold(4)
        try:
            rows.attend(q, kv, entry, SCALE, stream=streams[failing])
        finally:
            ula.ula_rows_debug_hold(-1)
        torch.cuda.synchronize()
        for s in streams:
            with pytest.raises(ula.UlaError) as e:
                rows.sync(s)
            assert e.value.code == ula.ERR_TIMEOUT
        for s in streams:
            rows.sync(s)


def test_rotate_output_over_itself():
    """An output whose tokens or heads share memory is refused; one that interleaves is not."""
    from serving_step_sparse_gb300 import rows, ula
    rng = np.random.default_rng(8)
    rot, _, _ = make_rotary(rng, 1, "halves")
    x = torch.from_numpy(rng.standard_normal((6, 4, 64))).float().cuda()
    pos = torch.from_numpy(positions(rng, 1, 6)).cuda()
    want = rows.rotate(x, pos, rot)
    store = torch.zeros(6 * 4 * 64 + 64, device="cuda")
    for shape, stride in (((6, 4, 64), (0, 64, 1)), ((6, 4, 64), (256, 0, 1)), ((6, 4, 64), (192, 64, 1)),
                          ((6, 4, 64), (64, 320, 1)), ((6, 4, 64), (256, 32, 1))):
        with pytest.raises(ula.UlaError) as e:
            rows.rotate(x, pos, rot, out=store.as_strided(shape, stride))
        assert e.value.code == ula.ERR_INVALID_ARG
    assert not store.any()
    for stride in ((256, 64, 1), (64, 384, 1)):
        out = torch.zeros(4 * 384, device="cuda").as_strided((6, 4, 64), stride)
        assert torch.equal(rows.rotate(x, pos, rot, out=out), want)


def test_tensors_that_require_a_gradient():
    """They are refused where a gradient would be recorded."""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(17)
    rot, _, _ = make_rotary(rng, 1, "halves")
    x = torch.from_numpy(rng.standard_normal((5, 2, 64))).float().cuda()
    pos = torch.from_numpy(positions(rng, 1, 5)).cuda()
    want = rows.rotate(x, pos, rot)
    for args in ((x.clone().requires_grad_(), None), (x, torch.zeros_like(x).requires_grad_() * 1)):
        with pytest.raises(ValueError, match="gradient"):
            rows.rotate(args[0], pos, rot, out=args[1])
        with torch.no_grad():
            assert torch.equal(rows.rotate(args[0], pos, rot, out=args[1]), want)


def test_outputs_handed_in_count_as_written():
    """Autograd notices a saved tensor that a call has changed."""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(18)
    rot, _, _ = make_rotary(rng, 1, "halves")
    x = torch.from_numpy(rng.standard_normal((5, 2, 64))).float().cuda()
    pos = torch.from_numpy(positions(rng, 1, 5)).cuda()
    want = rows.rotate(x, pos, rot)
    w = torch.ones(5, 2, 64, device="cuda", requires_grad=True)
    y = x.clone()
    loss = (w * y).sum()                                    # y is saved for w's gradient
    rows.rotate(y, pos, rot, out=y)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    q, kv, entry, own_rows = attend_case(1, 2, 8, 20, 20, 5, own=True)
    o, z = rows.attend(q, kv, entry, SCALE)
    tensors = (o, z, own_rows, q, kv, entry)
    before = [t._version for t in tensors]
    rows.attend(q, kv, entry, SCALE, out=o, lse=z)
    rows.join([o], [z], out=o, lse=z)
    rows.pack(torch.zeros(1, 512, device="cuda"), torch.zeros(1, 64, device="cuda"),
              torch.zeros(1, dtype=torch.int32, device="cuda"), rot, own_rows[0, :1])
    assert [t._version - b for t, b in zip(tensors, before)] == [2, 2, 1, 0, 0, 0]
    with torch.inference_mode():
        y = x.clone()
        assert torch.equal(rows.rotate(y, pos, rot, out=y), want)


def test_strides_of_single_elements():
    """The stride of a dimension of one element says nothing: no reason to refuse a call."""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(23)

    def odd(t, dims):
        return t.as_strided(t.shape, [3 if d in dims else s for d, s in enumerate(t.stride())])

    q, kv, entry, own_rows = attend_case(1, 3, 20, 40, 30, 2, own=True)
    want = rows.attend(q, kv, entry, SCALE, own_rows=own_rows)
    got = rows.attend(odd(q, [0]), kv, odd(entry, [0]), SCALE, own_rows=odd(own_rows, [0]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q, kv, entry, own_rows = attend_case(3, 1, 1, 40, 30, 2, own=True)
    want = rows.attend(q, kv, entry, SCALE, own_rows=own_rows)
    got = rows.attend(odd(q, [1, 2]), kv, odd(entry, [1]), SCALE, own_rows=odd(own_rows, [1]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    rot, _, _ = make_rotary(rng, 1, "halves")
    x = torch.from_numpy(rng.standard_normal((1, 4, 64))).to(torch.bfloat16).cuda()
    pos = torch.tensor([[5]], dtype=torch.int32, device="cuda")
    want = rows.rotate(x, pos, rot)
    assert torch.equal(rows.rotate(odd(x, [0]), pos, rot, out=odd(torch.zeros_like(x), [0])), want)
    latent, rope = x.flatten()[None, :].repeat(1, 2)[:, :512], x[:, 0]
    want = rows.pack(latent, rope, pos, rot)
    assert torch.equal(rows.pack(odd(latent, [0]), odd(rope, [0]), pos, rot, odd(torch.zeros_like(want), [0])), want)


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_rotate_same_bits_at_any_alignment(dtype, pairing):
    """What an output holds does not depend on how its memory lies, nor on the kernel that
    this chooses; a row's rope channels are the rotation's."""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(29)
    rot, _, _ = make_rotary(rng, 3, pairing)
    x = torch.from_numpy(rng.standard_normal((501, 9, 64))).to(DT[dtype]).cuda()
    pos = torch.from_numpy(positions(rng, 3, 501)).cuda()
    for inverse in (False, True):
        want = rows.rotate(x, pos, rot, inverse=inverse)
        for at in (0, 1, 2, 8):
            odd = torch.zeros(501, 9, 73, dtype=DT[dtype], device="cuda")[..., at:at + 64]
            assert torch.equal(rows.rotate(x, pos, rot, out=odd, inverse=inverse), want)
    packed = rows.pack(torch.zeros(501, 512, dtype=DT[dtype], device="cuda"), x[:, 0], pos, rot)
    if dtype != "f16":                                      # (rows hold bf16, rounded once)
        assert torch.equal(packed[:, 528:].contiguous().view(torch.bfloat16),
                           rows.rotate(x[:, 0], pos, rot).to(torch.bfloat16))


# ------------------------------------------------------------------------------- many rows

def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("heads,more", [(8, 1), (37, 5), (129, 700), (3, 0), (1, 3)])
def test_rotate_many(heads, more, dtype, pairing):
    """Prompt sizes: from 2 x 4 blocks' rows for every SM on, threads take two rows each (tokens
    of fewer than 8 heads excepted); the last block has a remainder."""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(heads + more)
    step = 32 if dtype == "f32" else 64                     # rows a block takes at once
    n = -(-8 * step * sms() // heads) + more
    rot, freq, axis = make_rotary(rng, 2, pairing)
    x = torch.from_numpy(rng.standard_normal((n, heads, 64), dtype=np.float32)).to(DT[dtype]).cuda()
    pos = positions(rng, 2, n)
    pos_d = torch.from_numpy(pos).cuda()
    out = rows.rotate(x, pos_d, rot)
    check_turned(out, x.double().cpu(), pos, freq, axis, pairing, dtype)
    back = rows.rotate(x, pos_d, rot, inverse=True)
    check_turned(back, x.double().cpu(), pos, freq, axis, pairing, dtype, sign=-1.0)
    wide = torch.full((n, heads, 80), 7.0, dtype=DT[dtype], device="cuda")
    wide[..., 8:72] = x
    rows.rotate(wide[..., 8:72], pos_d, rot, out=wide[..., 8:72])                  # in place, strided
    assert torch.equal(wide[..., 8:72], out)
    assert (wide[..., :8] == 7).all() and (wide[..., 72:] == 7).all()
    odd = torch.zeros(n, heads, 65, dtype=DT[dtype], device="cuda")                # unaligned rows
    assert torch.equal(rows.rotate(x, pos_d, rot, out=odd[..., 1:]), out)


def check_packed(got, latent, rope, pos, freq, axis, pairing):
    """As test_pack has it."""
    n = latent.shape[0]
    b = got.cpu().numpy()
    v = latent.double().cpu().numpy().reshape(n, 4, 128)
    scale = np.ascontiguousarray(b[:, 512:528]).view(np.float32).astype(np.float64)
    want = np.maximum(np.abs(v).max(-1) / 448, 2.0 ** -126)
    assert (np.abs(scale - want) <= 2.0 ** -23 * want).all()
    codes = E4M3[b[:, :512]].reshape(n, 4, 128)
    y = v / scale[..., None]
    spacing = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))) - 3)
    assert (np.abs(codes - y) <= spacing / 2 + 2.0 ** -21 * np.abs(y)).all()
    got_rope = torch.from_numpy(np.ascontiguousarray(b[:, 528:])).view(torch.bfloat16)
    check_turned(got_rope, rope.double().cpu(), pos, freq, axis, pairing, "bf16")


@pytest.mark.parametrize("pairing", ["adjacent", "halves"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rounds,more", [(1, 0), (1, 1), (2, -3), (2, 270), (4, 9)])
def test_pack_many(rounds, more, dtype, pairing):
    """Document sizes: a warp takes more than one token past 4 blocks of 8 warps for every SM."""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(rounds * 17 + more)
    n = rounds * 32 * sms() + more
    rot, freq, axis = make_rotary(rng, 3, pairing)
    x = rng.standard_normal((n, 576), dtype=np.float32) * np.exp(rng.standard_normal((n, 1), dtype=np.float32))
    pos = positions(rng, 3, n)
    pos_d = torch.from_numpy(pos).cuda()
    both = torch.from_numpy(x).to(DT[dtype]).cuda()
    dest = torch.full((n, 2, 656), 0xA5, dtype=torch.uint8, device="cuda")
    got = rows.pack(both[:, :512], both[:, 512:], pos_d, rot, dest[:, 1])
    assert (dest[:, 0] == 0xA5).all()
    check_packed(got, both[:, :512], both[:, 512:], pos, freq, axis, pairing)
    odd = torch.zeros(n, 577, dtype=DT[dtype], device="cuda")                      # unaligned latents
    odd[:, 1:] = both
    assert torch.equal(rows.pack(odd[:, 1:513], odd[:, 513:], pos_d, rot), got)


# ------------------------------------------------------------------------------- with the cache

@pytest.mark.parametrize("R,Q,H,K", [(1, 129, 8, 40), (2, 300, 20, 7), (1, 200, 64, 0), (3, 140, 3, 120), (1, 260, 128, 200)])
def test_attend_own_rows_over_tiles(R, Q, H, K):
    """A chunk of a prompt: more query tokens than a tile has rows, each of which sees the own
    rows up to itself, behind lists that end inside a tile."""
    from serving_step_sparse_gb300 import rows
    q, kv, entry, own_rows = attend_case(R, Q, H, K, 200, R + Q + H, pads=0.1, own=True)
    got = rows.attend(q, kv, entry, SCALE, own_rows=own_rows)
    check_attend(got, attend64(q, kv, entry, SCALE, own_rows))
    bad = own_rows.clone()                                  # a token's row is seen by later ones only
    bad[0, Q // 2, 512:528] = torch.tensor([math.nan] * 4).view(torch.uint8).cuda()
    out, lse = rows.attend(q, kv, entry, SCALE, own_rows=bad)
    assert torch.equal(out[0, :Q // 2], got[0][0, :Q // 2]) and torch.equal(lse[0, :Q // 2], got[1][0, :Q // 2])
    assert torch.isnan(out[0, Q // 2:]).all() and torch.isnan(lse[0, Q // 2:]).all()
    rows.sync()


def layer_rows(n, layers, rng):
    """[n][layers][656]: rows for the cache, one group."""
    return random_rows(n * layers, rng).view(n, layers, 656)


def test_attend_after_a_step_with_pads():
    """Selections with pads, as a request shorter than the top-k has them, through step_group."""
    from serving_step_sparse_gb300 import rows, ula
    from serving_step_sparse_gb300.cache import UlaCache
    rng = np.random.default_rng(41)
    R, Q, K, L, H, n = 3, 2, 96, 2, 20, 700
    store = layer_rows(n, L, rng)
    cache = UlaCache(row_bytes=656, layers_per_group=[L], gpu_slots=n // 2, host_slots=n, ring_buckets=4,
                     max_logical=n, max_entries=R * Q * K)
    try:
        assert cache.alloc(n, store) == 0
        entry_row = torch.empty(R * Q * K, dtype=torch.int32, device="cuda")
        req_off = torch.empty(R + 1, dtype=torch.int32, device="cuda")
        for step in range(3):
            sel = np.stack([[rng.choice(200, K, replace=False) + 230 * r for _ in range(Q)] for r in range(R)])
            sel[0, :, 10 + step:] = -1                      # a short request: pads behind
            sel[1][rng.random((Q, K)) < 0.4] = -1           # pads anywhere
            sel[2, 1] = -1                                  # a token that selects nothing
            sel = torch.from_numpy(sel.astype(np.int32)).cuda()
            assert int(sel.min()) == -1 and ula.ADDR_PAD == 2 ** 32 - 1
            out = cache.out_buffer(0, R * Q * K)
            out.fill_(0xFF)                                 # (NaN where nothing is gathered)
            cache.step_group(0, sel, out, entry_row, req_off)
            q = attend_case(R, Q, H, 1, 1, 400 + step)[0]
            for j in range(L):
                got = rows.attend(q, out[j], entry_row.view(R, Q, K), SCALE)
                check_attend(got, attend64(q, store[:, j].contiguous(), sel, SCALE))
        cache.sync()
        rows.sync()
    finally:
        cache.close()


@pytest.mark.parametrize("parts", [2, 4])
def test_attend_after_a_tp_step(parts):
    """What a UlaTP step leaves each rank, its local rows and the remote ones with an entry list
    for each, attended to separately and joined, against all rows at once."""
    from serving_step_sparse_gb300 import rows
    from serving_step_sparse_gb300.cache import UlaTP
    rng = np.random.default_rng(43 + parts)
    R, Q, K, L, H, n = 2, 3, 150, 2, 24, 2400
    E = R * Q * K
    store = layer_rows(n, L, rng)
    tp = UlaTP(row_bytes=656, layers_per_group=[L], parts=parts, gpu_slots=3 * n // (4 * parts), host_slots=n,
               ring_buckets=4, max_logical=n, max_entries=E, buffer_slots=2 * E)
    try:
        assert tp.alloc(n, store) == 0
        tp.sync()
        of_rank = lambda size: [torch.empty(size, dtype=torch.int32, device="cuda") for _ in range(parts)]
        for step in range(2):
            # recent tokens of one partition only (nothing remote for one rank), pads, an empty token
            sel = np.stack([[rng.choice(1200, K, replace=False) + 1200 * r for _ in range(Q)] for r in range(R)])
            sel[0, 0] = parts * rng.choice(n // parts, K, replace=False)
            sel[1, 1, 40:] = -1
            sel[1, 2] = -1
            sel = torch.from_numpy(sel.astype(np.int32)).cuda()
            local, remote = ([tp.out_buffer(0, E).fill_(0xFF) for _ in range(parts)] for _ in range(2))
            local_row, remote_row, local_off, remote_off = of_rank(E), of_rank(E), of_rank(R + 1), of_rank(R + 1)
            tp.step_group(0, sel, local, remote, local_row, local_off, remote_row, remote_off)
            tp.sync()
            q = attend_case(R, Q, H, 1, 1, 500 + step)[0]
            for j in range(L):
                out, lse, slack, zslack = attend64(q, store[:, j].contiguous(), sel, SCALE)
                none = np.isneginf(lse)
                assert none.any() and not none.all()
                for r in range(parts):
                    a = rows.attend(q, local[r][j], local_row[r].view(R, Q, K), SCALE)
                    b = rows.attend(q, remote[r][j], remote_row[r].view(R, Q, K), SCALE)
                    o, z = rows.join([a[0], b[0]], [a[1], b[1]])
                    o, z = o.double().cpu().numpy(), z.double().cpu().numpy()
                    assert np.array_equal(np.isneginf(z), none) and (o[none] == 0).all()
                    assert (np.abs(z[~none] - lse[~none]) <= (zslack + 2.0 ** -19 * (1 + np.abs(lse)))[~none]).all()
                    # each part was rounded to bf16 as well
                    tol = 2.0 ** -8 * 1.01 * np.abs(out) + (2.0 ** -8 + 2.0 ** -8 + np.expm1(2 * zslack[..., None])) * slack
                    assert (np.abs(o - out) <= tol)[~none].all()
        tp.sync()
        rows.sync()
    finally:
        tp.close()


@pytest.mark.parametrize("R,H,K", [(2, 20, 700), (12, 16, 1024), (160, 64, 150)])
def test_operators_in_a_graph(R, H, K):
    """A layer's calls captured once and replayed on new inputs give what the calls give."""
    from serving_step_sparse_gb300 import rows
    rng = np.random.default_rng(R)
    rot, _, _ = make_rotary(rng, 1, "halves")
    pos = torch.arange(R, dtype=torch.int32, device="cuda")
    cases = [attend_case(R, 1, H, K, 400, 70 + s, pads=0.1) for s in range(3)]
    new = [torch.from_numpy(rng.standard_normal((3, R, 576))).to(torch.bfloat16).cuda()[s] for s in range(3)]

    def layer(q, kv, entry, x):
        turned = q.clone()
        rope = turned.view(R, H, 576)[..., 512:]
        rows.rotate(rope, pos, rot, out=rope)
        own = rows.pack(x[:, :512], x[:, 512:], pos, rot).view(R, 1, 656)
        a = rows.attend(turned, kv, entry, SCALE, own_rows=own)
        b = rows.attend(turned, kv, entry.flip(-1)[..., :K // 3].contiguous(), SCALE)
        return rows.join([a[0], b[0]], [a[1], b[1]])

    want = [layer(*c[:3], x) for c, x in zip(cases, new)]
    held = [t.clone() for t in (*cases[0][:3], new[0])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(*held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(*held)
    for s in (1, 2, 0, 1):
        for h, t in zip(held, (*cases[s][:3], new[s])):
            h.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[s][0]) and torch.equal(got[1], want[s][1])
    rows.sync()
