"""Cases of the operators on the cache's FP8 rows: rotary positions, row packing, attention, joining.

A row is 656 bytes: 512 e4m3 latent channels, 4 fp32 scales (one per block of 128 channels) and
64 bf16 rope channels.  ``run`` computes a case in its plain form (elementary torch operations in
32 bits) or, where ``own`` is set, by the calls of ``serving_step_sparse_gb300.rows``; ``exact``
gives the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

LATENT, ROPE, BLOCK, ROW = 512, 64, 128, 656
BLOCKS = LATENT // BLOCK
PAIRS = ROPE // 2
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
SOFTMAX_SCALE = (128 + ROPE) ** -0.5
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------------------- the cases

def listed():
    def attend(name, req, q, heads, k, own_rows=False, pads=0.0, empty=False):
        return {"name": name, "op": "attend", "req": req, "q": q, "heads": heads, "k": k,
                "own_rows": own_rows, "pads": pads, "empty": empty}

    def rotate(name, tokens, heads, dtype, axes, pairing):
        return {"name": name, "op": "rotate", "tokens": tokens, "heads": heads, "dtype": dtype,
                "axes": axes, "pairing": pairing}

    def pack(name, tokens, layers, dtype, axes, pairing):
        return {"name": name, "op": "pack", "tokens": tokens, "layers": layers, "dtype": dtype,
                "axes": axes, "pairing": pairing}

    def join(name, parts, tokens, heads, empty):
        return {"name": name, "op": "join", "parts": parts, "tokens": tokens, "heads": heads,
                "empty": empty}

    return [
        # one request with a short selection (the tiny workload's 256 rows): latency
        attend("attend_one_request", 1, 1, 32, 256),
        # eight requests, one query token each (the batch workload's selection): few rows of queries
        attend("attend_batch8", 8, 1, 64, 2048),
        # requests shorter than the selection: pads, an odd length and head count, a query that
        # selects nothing at all
        attend("attend_ragged", 5, 2, 20, 777, pads=0.1, empty=True),
        # the long-document step of one layer: 3 query tokens a request, which also see their own
        # rows, with the heads of a model half as wide as the next case's
        attend("attend_longdoc_64", 32, 3, 64, 2048, own_rows=True),
        # the same with 128 heads: the largest product of a decode step
        attend("attend_longdoc_128", 32, 3, 128, 2048, own_rows=True),
        # a decode step's queries (32 requests x 3 tokens), text and image positions
        rotate("rotate_decode", 96, 64, "bf16", 3, "halves"),
        # the queries of a prompt chunk
        rotate("rotate_prompt", 4096, 128, "bf16", 1, "adjacent"),
        # a decode step's new tokens, one layer of four in a group
        pack("pack_decode", 96, 4, "bf16", 3, "halves"),
        # an odd chunk of a prompt with frames, from 32-bit activations
        pack("pack_chunk_odd", 4097, 4, "f32", 3, "adjacent"),
        # one layer of a whole long document
        pack("pack_document", 131072, 1, "bf16", 1, "adjacent"),
        # two partitions' partial results of a decode step
        join("join_two_parts", 2, 96, 64, False),
        # a few queries, parts that found nothing
        join("join_few_odd", 3, 7, 20, True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.4)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "attend", "rotate", "pack", "pack", "join"])
    pairing = rng.choice(["adjacent", "halves"])
    axes = rng.choice([1, 2, 3, 4])
    if op == "attend":
        while True:
            case = {"op": op, "req": _log_int(rng, 1, 64), "q": rng.randint(1, 4),
                    "heads": _log_int(rng, 1, 128), "k": _log_int(rng, 1, 4096),
                    "own_rows": rng.random() < 0.5, "pads": rng.choice([0.0, 0.0, 0.1, 0.6]),
                    "empty": rng.random() < 0.3}
            rows = case["req"] * case["q"] * case["k"]
            if rows <= 96 * 2048 and rows * case["heads"] <= 96 * 2048 * 128:
                return case
    if op == "rotate":
        while True:
            case = {"op": op, "tokens": _log_int(rng, 1, 8192), "heads": _log_int(rng, 1, 128),
                    "dtype": rng.choice(["bf16", "bf16", "f16"]), "axes": axes, "pairing": pairing}
            if case["tokens"] * case["heads"] <= 4096 * 128:
                return case
    if op == "pack":
        while True:
            case = {"op": op, "tokens": _log_int(rng, 1, 131072), "layers": rng.choice([1, 3, 4]),
                    "dtype": rng.choice(["bf16", "f16", "f32"]), "axes": axes, "pairing": pairing}
            if case["tokens"] * case["layers"] <= 131072 and (
                    case["dtype"] != "f32" or case["tokens"] <= 65536):
                return case
    return {"op": "join", "parts": rng.randint(2, 8), "tokens": _log_int(rng, 1, 192),
            "heads": _log_int(rng, 1, 128), "empty": rng.random() < 0.4}


# ------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _quantise_rows(x, rope):
    """Cache rows as another program would have stored them: x [n][512], rope [n][64] -> [n][656]."""
    n = x.shape[0]
    blocks = x.view(n, BLOCKS, BLOCK)
    scale = (blocks.abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN)
    codes = (blocks / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.cat([codes.view(n, LATENT), scale.view(torch.uint8).view(n, 4 * BLOCKS),
                      rope.to(torch.bfloat16).view(torch.uint8).view(n, 2 * ROPE)], dim=1)


def _cache_rows(g, n):
    # latents after a norm: unit size, some channels and some tokens larger than others
    x = _randn(g, n, LATENT) * torch.exp(0.3 * _randn(g, 1, LATENT)) * torch.exp(0.2 * _randn(g, n, 1))
    return _quantise_rows(x, _randn(g, n, ROPE))


def _rotary(case):
    """Frequencies of the 32 pairs (base 10,000) and the axis of each: one axis for text; time,
    height, width (and one more) in consecutive sections otherwise."""
    freq = [float(torch.tensor(10000.0 ** (-j / PAIRS), dtype=torch.float32)) for j in range(PAIRS)]
    a = case["axes"]
    axis = [min(a - 1, j * a // PAIRS) for j in range(PAIRS)]
    return freq, axis


def _positions(case, g, n):
    """[axes][n]: the running position (documents up to 131,072 tokens) and grid positions."""
    start = int(torch.randint(0, max(1, 131072 - n), (1,), generator=g, device="cuda"))
    pos = torch.randint(0, 256, (case["axes"], n), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = torch.arange(start, start + n, device="cuda", dtype=torch.int32)
    return pos


def _distinct(case):
    """Distinct rows that one request's query tokens select together (nine tenths are shared)."""
    return case["k"] + (case["q"] - 1) * (case["k"] // 10)


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": dict(case)}
    if op == "attend":
        R, Q, H, K = case["req"], case["q"], case["heads"], case["k"]
        nu = _distinct(case)
        s["rows"] = _cache_rows(g, R * nu)
        s["q"] = _randn(g, R, Q, H, LATENT + ROPE).to(torch.bfloat16)
        # the gathered rows follow the first query token's order; later ones mix in fresh rows
        order = torch.rand(R, Q, nu, generator=g, device="cuda")
        order[:, 0] = torch.arange(nu, device="cuda") / max(1, nu)
        pick = order.argsort(-1)[..., :K].sort(-1).values.to(torch.int32)
        entry = pick + (torch.arange(R, device="cuda", dtype=torch.int32) * nu)[:, None, None]
        if case["pads"]:
            drop = torch.rand(R, Q, K, generator=g, device="cuda") < case["pads"]
            entry = torch.where(drop, torch.full_like(entry, -1), entry)
        if case["empty"]:
            entry[R // 2, Q - 1] = -1
        s["entry"] = entry.contiguous()
        s["own"] = _cache_rows(g, R * Q).view(R, Q, ROW) if case["own_rows"] else None
    elif op == "rotate":
        T, H = case["tokens"], case["heads"]
        s["x"] = _randn(g, T, H, ROPE).to(DTYPES[case["dtype"]])
        s["pos"] = _positions(case, g, T)
        # the rope part of the queries that the attention reads
        s["out"] = torch.zeros(T, H, LATENT + ROPE, dtype=DTYPES[case["dtype"]],
                               device="cuda")[..., LATENT:]
    elif op == "pack":
        T, L = case["tokens"], case["layers"]
        dt = DTYPES[case["dtype"]]
        s["latent"] = (_randn(g, T, LATENT) * torch.exp(0.3 * _randn(g, 1, LATENT))).to(dt)
        s["rope"] = _randn(g, T, ROPE).to(dt)
        s["pos"] = _positions(case, g, T)
        s["rows"] = torch.zeros(T, L, ROW, dtype=torch.uint8, device="cuda")[:, L - 1]
    else:
        P, T, H = case["parts"], case["tokens"], case["heads"]
        s["outs"] = [_randn(g, T, H, LATENT).to(torch.bfloat16) for _ in range(P)]
        s["lses"] = [6.0 + 2.0 * _randn(g, T, H) for _ in range(P)]
        if case["empty"]:
            for p in range(P):  # a part without rows for a query, and a query without any
                none = torch.rand(T, H, generator=g, device="cuda") < 0.3
                none[T // 2] = True
                s["lses"][p][none] = -math.inf
                s["outs"][p][none] = 0
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] in ("rotate", "pack"):
        freq, axis = _rotary(case)
        s["freq"], s["axis"] = freq, axis
        s["freq_t"] = torch.tensor(freq, device="cuda")
        s["axis_t"] = torch.tensor(axis, device="cuda")
    return s


# ------------------------------------------------------------------------------- the calls

def run(state):
    op = state["case"]["op"]
    if own:
        return {"attend": _own_attend, "rotate": _own_rotate, "pack": _own_pack,
                "join": _own_join}[op](state)
    return {"attend": _plain_attend, "rotate": _plain_rotate, "pack": _plain_pack,
            "join": _plain_join}[op](state)


def _own_attend(s):
    from serving_step_sparse_gb300 import rows
    return rows.attend(s["q"], s["rows"], s["entry"], SOFTMAX_SCALE, own_rows=s["own"])


def _own_rotary(s):
    from serving_step_sparse_gb300 import rows
    if "rotary" not in s:  # kept by a program from layer to layer and step to step
        s["rotary"] = rows.Rotary(s["freq"], s["axis"], s["case"]["pairing"])
    return s["rotary"]


def _own_rotate(s):
    from serving_step_sparse_gb300 import rows
    return rows.rotate(s["x"], s["pos"], _own_rotary(s), out=s["out"])


def _own_pack(s):
    from serving_step_sparse_gb300 import rows
    return _parts_of(rows.pack(s["latent"], s["rope"], s["pos"], _own_rotary(s), s["rows"]))


def _own_join(s):
    from serving_step_sparse_gb300 import rows
    return rows.join(s["outs"], s["lses"])


def _parts_of(rows):
    """A row's three parts as what they hold (views)."""
    return {"codes": rows[:, :LATENT].view(torch.float8_e4m3fn),
            "scales": rows.view(torch.float32)[:, LATENT // 4:LATENT // 4 + BLOCKS],
            "rope": rows.view(torch.bfloat16)[:, (LATENT + 4 * BLOCKS) // 2:]}


def _plain_attend(s):
    q, rows, entry, own_rows = s["q"], s["rows"], s["entry"], s["own"]
    R, Q, H, _ = q.shape
    valid = entry >= 0
    picked = rows[entry.clamp_min(0).long()]
    if own_rows is not None:  # query token i of a request sees its own rows 0..i
        picked = torch.cat([picked, own_rows[:, None].expand(R, Q, Q, ROW)], dim=2)
        seen = torch.ones(Q, Q, dtype=torch.bool, device=q.device).tril()
        valid = torch.cat([valid, seen.expand(R, Q, Q)], dim=2)
    codes = picked[..., :LATENT].contiguous().view(torch.float8_e4m3fn).float()
    scales = picked[..., LATENT:LATENT + 4 * BLOCKS].contiguous().view(torch.float32)
    rope = picked[..., LATENT + 4 * BLOCKS:].contiguous().view(torch.bfloat16).float()
    latent = (codes.unflatten(-1, (BLOCKS, BLOCK)) * scales[..., None]).flatten(-2)
    keys = torch.cat([latent, rope], dim=-1)
    logits = torch.matmul(q.float(), keys.transpose(-1, -2)) * SOFTMAX_SCALE
    logits = logits.masked_fill(~valid[:, :, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(torch.isneginf(top), torch.zeros_like(top), top)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, latent) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).squeeze(-1)
    return out.to(torch.bfloat16), lse


def _plain_turn(s, x):
    """Rotates the pairs of x [n][...][64] by the angle of each pair's axis; 32 bits."""
    angle = s["pos"].float()[s["axis_t"]].t() * s["freq_t"]      # [n][32]
    angle = angle.view(angle.shape[0], *([1] * (x.dim() - 2)), PAIRS)
    c, w = torch.cos(angle), torch.sin(angle)
    x = x.float()
    if s["case"]["pairing"] == "adjacent":
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * w, a * w + b * c], dim=-1).flatten(-2)
    a, b = x[..., :PAIRS], x[..., PAIRS:]
    return torch.cat([a * c - b * w, a * w + b * c], dim=-1)


def _plain_rotate(s):
    s["out"].copy_(_plain_turn(s, s["x"]))
    return s["out"]


def _plain_pack(s):
    s["rows"].copy_(_quantise_rows(s["latent"].float(), _plain_turn(s, s["rope"])))
    return _parts_of(s["rows"])


def _plain_join(s):
    outs, lses = torch.stack(s["outs"]).float(), torch.stack(s["lses"])
    top = lses.amax(0)
    top = torch.where(torch.isneginf(top), torch.zeros_like(top), top)
    w = torch.exp(lses - top)
    total = w.sum(0)
    out = (outs * w[..., None]).sum(0) / torch.where(total == 0, torch.ones_like(total), total)[..., None]
    return out.to(torch.bfloat16), top + torch.log(total)


# ------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "attend":
        T, H, K = case["req"] * case["q"], case["heads"], case["k"]
        keep = 1.0 - case["pads"]
        rows = case["req"] * _distinct(case) * min(1.0, keep * case["q"])
        own_keys = case["req"] * case["q"] * (case["q"] + 1) / 2 if case["own_rows"] else 0
        keys = T * K * keep + own_keys
        bytes_ = (T * H * (LATENT + ROPE) * 2 + T * H * LATENT * 2 + T * H * 4 + T * K * 4
                  + (rows + (T if case["own_rows"] else 0)) * ROW)
        return {"bytes": bytes_, "flops": 2.0 * keys * H * (2 * LATENT + ROPE)}
    if op == "rotate":
        n = case["tokens"] * case["heads"] * ROPE
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": 2 * n * size + 4 * case["axes"] * case["tokens"], "flops": 3.0 * n}
    if op == "pack":
        size = 4 if case["dtype"] == "f32" else 2
        t = case["tokens"]
        return {"bytes": t * ((LATENT + ROPE) * size + ROW + 4 * case["axes"]),
                "flops": t * (3.0 * LATENT + 3.0 * ROPE)}
    n = case["tokens"] * case["heads"]
    return {"bytes": (case["parts"] + 1) * n * (LATENT * 2 + 4),
            "flops": 2.0 * case["parts"] * n * LATENT}


# ------------------------------------------------------------------------------- 64 bits

def _e4m3_table():
    """The 256 values of e4m3 from its definition: sign, 4 exponent bits (bias 7), 3 mantissa bits,
    0x7f and 0xff not a number."""
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        v.append(math.nan if (b & 127) == 127 else -x if b & 128 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _unpack64(rows):
    n = rows.shape[0]
    lat = _e4m3_table()[rows[:, :LATENT].long()]
    sc = rows[:, LATENT:LATENT + 16].contiguous().view(torch.float32).double()
    rope = rows[:, LATENT + 16:].contiguous().view(torch.bfloat16).double()
    return lat * sc.repeat_interleave(BLOCK, dim=1), rope.view(n, ROPE)


def _turn64(case, pos, x):
    freq, axis = _rotary(case)
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for j in range(PAIRS):
        ang = pos[axis[j]].double() * freq[j]
        ang = ang.view(-1, *([1] * (x.dim() - 2)))
        i0, i1 = (2 * j, 2 * j + 1) if case["pairing"] == "adjacent" else (j, j + PAIRS)
        u, v = x[..., i0].double(), x[..., i1].double()
        out[..., i0] = u * torch.cos(ang) - v * torch.sin(ang)
        out[..., i1] = v * torch.cos(ang) + u * torch.sin(ang)
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "attend":
        R, Q, H, _ = s["q"].shape
        out = torch.zeros(R, Q, H, LATENT, dtype=torch.float64, device="cuda")
        lse = torch.full((R, Q, H), -math.inf, dtype=torch.float64, device="cuda")
        for r in range(R):
            for i in range(Q):
                idx = s["entry"][r, i]
                picked = s["rows"][idx[idx >= 0].long()]
                if s["own"] is not None:
                    picked = torch.cat([picked, s["own"][r, :i + 1]])
                if picked.shape[0] == 0:
                    continue
                lat, rope = _unpack64(picked)
                qd = s["q"][r, i].double()
                z = (qd[:, :LATENT] @ lat.t() + qd[:, LATENT:] @ rope.t()) * SOFTMAX_SCALE
                lse[r, i] = torch.logsumexp(z, dim=1)
                out[r, i] = torch.softmax(z, dim=1) @ lat
        return out, lse
    if op == "rotate":
        return _turn64(case, s["pos"], s["x"])
    if op == "pack":
        x = s["latent"].double()
        n = x.shape[0]
        scale = (x.view(n, BLOCKS, BLOCK).abs().amax(-1) / E4M3_MAX).clamp_min(SCALE_MIN)
        y = (x.view(n, BLOCKS, BLOCK) / scale[..., None]).view(n, LATENT)
        # the nearest e4m3 value: spacing 2^(e-3), 2^-9 at the least; halves go to the even one
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
        codes = (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
        return {"codes": codes, "scales": scale, "rope": _turn64(case, s["pos"], s["rope"])}
    z = torch.stack([x.double() for x in s["lses"]])
    o = torch.stack([x.double() for x in s["outs"]])
    lse = torch.logsumexp(z, dim=0)
    w = torch.exp(z - lse)
    w = torch.where(torch.isneginf(lse).expand_as(w), torch.zeros_like(w), w)
    return (o * w[..., None]).sum(0), lse
