"""The operators of a drafted step without a GPU: constants against the header, and refusals made on the host."""
import ctypes as C
import math
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ula.h")


@pytest.fixture(scope="module")
def ula():
    from serving_step_sparse_gb300.build import build
    build()
    from serving_step_sparse_gb300 import ula
    return ula


class AttendArgs(C.Structure):
    _fields_ = [("q", C.c_void_p), ("q_strides", C.c_uint64 * 3), ("rows", C.c_void_p), ("entry_row", C.c_void_p),
                ("own_rows", C.c_void_p), ("own_strides", C.c_uint64 * 2), ("out", C.c_void_p), ("lse", C.c_void_p),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_uint64)] + [
        (n, C.c_uint32) for n in ("n_rows", "n_req", "n_q", "heads", "k")] + [("scale", C.c_float)]


class ScoreArgs(C.Structure):
    _fields_ = [("q", C.c_void_p), ("q_strides", C.c_uint64 * 3)] + [
        (n, C.c_void_p) for n in ("rows", "entry_row", "address", "lse", "scores", "workspace")] + [
        ("workspace_bytes", C.c_uint64)] + [
        (n, C.c_uint32) for n in ("n_rows", "n_scores", "n_req", "n_q", "heads", "k", "flags")] + [("scale", C.c_float)]


def test_constants_match_header(ula):
    src = open(HEADER).read()
    for name, val in (("ULA_MAX_TREE", 64), ("ULA_TREE_SHARED_LIST", 1), ("ULA_MAX_WIDTH", 1024)):
        assert int(re.search(rf"#define {name} (\d+)u", src).group(1)) == val, name
    barriers = int(re.search(r"#define ULA_DEBUG_SCORE_BARRIERS (\d+)", src).group(1))
    for bad in (barriers, 10 ** 6):
        with pytest.raises(ula.UlaError):
            ula.ula_rows_debug_hold_score(bad)
    ula.ula_rows_debug_hold_score(barriers - 1)
    ula.ula_rows_debug_hold_score(-1)


def test_calls_refuse_on_the_host(ula):
    lib, none, u32, u64 = ula.lib, C.c_void_p(), C.c_uint32, C.c_uint64
    bad = ula.ERR_INVALID_ARG
    assert lib.ula_rows_attend_tree(none, none, u32(0), none) == bad
    assert lib.ula_rows_score(none, none) == bad
    rot = ula.ula_rotary(1, 0)
    at = C.c_void_p(1 << 20)  # (an address that is never read: every call below is refused, or has nothing to do)

    def norm(width=128, start=64, dtype=0, weight_dtype=0, eps=1e-6, n=1, heads=1, out_head=128, x=at):
        return lib.ula_rows_norm_rotate(C.byref(rot), at, u64(0), u32(n), u32(heads), u32(width), u32(start), u32(dtype), x, u64(0),
                                        u64(0), at, u32(weight_dtype), C.c_float(eps), at, u64(0), u64(out_head), none)
    for kw in (dict(width=63), dict(width=1025), dict(start=65), dict(dtype=3), dict(weight_dtype=1), dict(eps=-1.0), dict(eps=math.nan),
               dict(eps=math.inf), dict(heads=2, out_head=127), dict(x=none), dict(x=C.c_void_p((1 << 20) + 1))):
        assert norm(**kw) == bad, kw
    assert norm(n=0) == ula.OK and norm(heads=0) == ula.OK

    def pack(n=1, weight=at, weight_dtype=0, rope_weight_dtype=0, eps=1e-6, stride=656, dtype=0):
        return lib.ula_rows_pack_norm(C.byref(rot), at, u64(0), u32(n), u32(dtype), at, u64(512), at, u64(64), weight, u32(weight_dtype),
                                      at, u32(rope_weight_dtype), C.c_float(eps), at, u64(stride), none)
    for kw in (dict(weight=none), dict(weight_dtype=1), dict(rope_weight_dtype=1), dict(eps=-1.0), dict(stride=640), dict(dtype=3)):
        assert pack(**kw) == bad, kw
    assert pack(n=0) == ula.OK

    def evict(n_req=1, longest=10, budget=4, first=1, last=1, scores=at, address=at, length=at, kept=at, dropped=at):
        return lib.ula_rows_evict(scores, u32(5), address, length, u32(n_req), u32(longest), u32(budget), u32(first), u32(last), kept,
                                  dropped, none)
    for kw in (dict(first=3, last=2), dict(longest=2 ** 31), dict(scores=none), dict(address=none), dict(length=none), dict(kept=none),
               dict(dropped=none), dict(kept=C.c_void_p((1 << 20) + 2))):
        assert evict(**kw) == bad, kw
    assert evict(n_req=0) == ula.OK


def tree_args(**kw):
    v = dict(q=1 << 20, rows=1 << 20, entry_row=1 << 20, own_rows=1 << 20, out=1 << 20, n_rows=9, n_req=2, n_q=3, heads=4, k=5)
    v.update(kw)
    a = AttendArgs(**{k: x for k, x in v.items() if k not in ("q_strides", "own_strides")})
    a.q_strides[:] = v.get("q_strides", [3 * 4 * 576, 4 * 576, 576])
    a.own_strides[:] = v.get("own_strides", [3 * 656, 656])
    return a


def test_tree_refuses_on_the_host(ula):
    lib, none, at, bad = ula.lib, C.c_void_p(), C.c_void_p(1 << 20), ula.ERR_INVALID_ARG
    call = lambda parent=at, flags=0, **kw: lib.ula_rows_attend_tree(C.byref(tree_args(**kw)), parent, C.c_uint32(flags), none)  # noqa: E731
    for kw in (dict(q=0), dict(out=0), dict(own_rows=0), dict(rows=0), dict(entry_row=0), dict(parent=none), dict(n_q=65), dict(flags=2),
               dict(parent=C.c_void_p((1 << 20) + 2)), dict(q=(1 << 20) + 8), dict(q_strides=[1, 4 * 576, 576]),
               dict(own_strides=[3 * 656, 8]), dict(heads=2 ** 26, flags=1), dict(k=2 ** 31)):
        assert call(**kw) == bad, kw
    for kw in (dict(n_req=0), dict(n_q=0), dict(heads=0)):
        assert call(**kw) == ula.OK, kw


def test_score_refuses_on_the_host(ula):
    lib, none, bad = ula.lib, C.c_void_p(), ula.ERR_INVALID_ARG
    lib.ula_rows_score_workspace.restype = C.c_uint64
    need = lib.ula_rows_score_workspace(2, 3, 4, 0, 100)

    def call(**kw):
        v = dict(q=1 << 20, rows=1 << 20, entry_row=1 << 20, address=1 << 20, lse=1 << 20, scores=1 << 20, workspace=1 << 20,
                 workspace_bytes=need, n_rows=9, n_scores=100, n_req=2, n_q=3, heads=4, k=5, flags=0)
        v.update(kw)
        a = ScoreArgs(**{k: x for k, x in v.items() if k != "q_strides"})
        a.q_strides[:] = v.get("q_strides", [3 * 4 * 576, 4 * 576, 576])
        return lib.ula_rows_score(C.byref(a), none)
    for kw in (dict(q=0), dict(rows=0), dict(entry_row=0), dict(address=0), dict(lse=0), dict(scores=0), dict(workspace=0), dict(flags=2),
               dict(workspace_bytes=need - 1), dict(workspace=(1 << 20) + 8), dict(q_strides=[3 * 4 * 576, 4, 576]), dict(scores=(1 << 20) + 2),
               dict(n_rows=2 ** 31), dict(n_scores=2 ** 31, workspace_bytes=2 ** 40), dict(k=2 ** 31)):
        assert call(**kw) == bad, kw
    for kw in (dict(n_req=0), dict(n_q=0), dict(heads=0), dict(k=0), dict(n_scores=0)):
        assert call(**kw) == ula.OK, kw


def test_host_tensors_are_refused(ula):
    from serving_step_sparse_gb300 import rows
    rot = rows.Rotary([1.0 / (j + 1) for j in range(32)])
    pos = torch.zeros(2, dtype=torch.int32)
    q, kv = torch.zeros(1, 2, 1, 576, dtype=torch.bfloat16), torch.zeros(4, 656, dtype=torch.uint8)
    entry, own = torch.zeros(1, 2, 4, dtype=torch.int32), torch.zeros(1, 2, 656, dtype=torch.uint8)
    for f in (lambda: rows.norm_rotate(torch.zeros(2, 64), torch.ones(64), pos, rot),
              lambda: rows.pack_norm(torch.zeros(2, 512), torch.zeros(2, 64), torch.ones(512), pos, rot),
              lambda: rows.attend_tree(q, kv, entry, 0.1, own, torch.zeros(1, 2, dtype=torch.int32)),
              lambda: rows.score(torch.zeros(9), q, kv, entry, entry, torch.zeros(1, 2, 1), 0.1),
              lambda: rows.evict(torch.zeros(9), entry[0], torch.zeros(2, dtype=torch.int32), 2)):
        with pytest.raises(ValueError):
            f()


def test_free_each_merges_runs(monkeypatch):
    """One call for each run of neighbours, pads left out."""
    from serving_step_sparse_gb300.cache import UlaCache
    cache, calls = UlaCache.__new__(UlaCache), []
    monkeypatch.setattr(UlaCache, "free", lambda self, base, n: calls.append((base, n)))
    cache.free_each(torch.tensor([[5, 4, -1], [9, 6, 20]], dtype=torch.int32))
    cache.free_each(torch.tensor([-1, -1], dtype=torch.int32))
    assert calls == [(4, 3), (9, 1), (20, 1)]


def test_evict_refuses_shared_memory(ula):
    """Outputs that lie in an input or in each other, by their last or first element."""
    lib, none, bad = ula.lib, C.c_void_p(), ula.ERR_INVALID_ARG
    at = dict(scores=1 << 20, address=2 << 20, length=3 << 20, kept=4 << 20, dropped=5 << 20)
    size = dict(scores=5, address=2 * 10, length=2, kept=2 * 4, dropped=2 * 6)

    def evict(**kw):
        v = {k: C.c_void_p(x) for k, x in {**at, **kw}.items()}
        return lib.ula_rows_evict(v["scores"], C.c_uint32(5), v["address"], v["length"], C.c_uint32(2), C.c_uint32(10), C.c_uint32(4),
                                  C.c_uint32(1), C.c_uint32(1), v["kept"], v["dropped"], none)
    for out in ("kept", "dropped"):
        for other in at:
            if other != out:
                for place in (at[other], at[other] + 4 * (size[other] - 1), at[other] - 4 * (size[out] - 1)):
                    assert evict(**{out: place}) == bad, (out, other, place)


def test_free_each_refuses_other_types():
    from serving_step_sparse_gb300.cache import UlaCache
    for wrong in (torch.zeros(2), torch.zeros(2, dtype=torch.bool), torch.zeros(2, dtype=torch.int16)):
        with pytest.raises(ValueError):
            UlaCache.__new__(UlaCache).free_each(wrong)


def test_tangents_are_refused(ula):
    """A dual tensor's tangent would be lost without a word, whichever argument it is."""
    import torch.autograd.forward_ad as fwd
    from serving_step_sparse_gb300 import rows
    rot = rows.Rotary([1.0 / (j + 1) for j in range(32)])
    pos = torch.zeros(2, dtype=torch.int32)
    x, latent, rope, w = torch.zeros(2, 64), torch.zeros(2, 512), torch.zeros(2, 64), torch.ones(512)
    q, kv = torch.zeros(1, 2, 1, 576, dtype=torch.bfloat16), torch.zeros(4, 656, dtype=torch.uint8)
    entry, own = torch.zeros(1, 2, 4, dtype=torch.int32), torch.zeros(1, 2, 656, dtype=torch.uint8)
    parent, lse, scores = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 2, 1), torch.zeros(9)
    length, out = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, 1, 512, dtype=torch.bfloat16)
    with fwd.dual_level():
        d = lambda t: fwd.make_dual(t, torch.ones_like(t))  # noqa: E731
        for f in (lambda: rows.rotate(d(x), pos, rot), lambda: rows.pack(d(latent), rope, pos, rot), lambda: rows.pack(latent, d(rope), pos, rot),
                  lambda: rows.norm_rotate(d(x), w[:64], pos, rot), lambda: rows.pack_norm(d(latent), rope, w, pos, rot),
                  lambda: rows.attend(d(q), kv, entry, 0.1), lambda: rows.attend_tree(d(q), kv, entry, 0.1, own, parent),
                  lambda: rows.join([d(out)], [lse]), lambda: rows.score(d(scores), q, kv, entry, entry, lse, 0.1),
                  lambda: rows.score(scores, d(q), kv, entry, entry, lse, 0.1), lambda: rows.evict(d(scores), entry[0], length, 2)):
            with pytest.raises(ValueError, match="tangent"):
                f()
    with pytest.raises(ValueError, match="device"):  # (outside: tensors as any others)
        rows.rotate(x, pos, rot)


def test_free_each_refuses_wide_addresses(monkeypatch):
    """2^32 + 5 is not address 5; nothing is freed."""
    from serving_step_sparse_gb300 import cache as module
    from serving_step_sparse_gb300.cache import UlaCache
    cache, calls = UlaCache.__new__(UlaCache), []
    cache.ctx = None
    monkeypatch.setattr(module.ula.lib, "ula_free", lambda ctx, base, n: calls.append((base, n)) or 0)
    for wide in (2 ** 32 + 5, 2 ** 32, 2 ** 62):
        with pytest.raises(ValueError):
            cache.free_each(torch.tensor([3, wide]))
    assert calls == []
    cache.free_each(torch.tensor([-(2 ** 40), 2 ** 32 - 1, 7]))
    assert calls == [(7, 1), (2 ** 32 - 1, 1)]
