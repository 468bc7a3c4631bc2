"""The operators on rows without a GPU: the binding against the header, and refusals that are
made on the host."""
import ctypes as C
import math
import os
import re
import subprocess

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


def test_constants_match_header(ula):
    src = open(HEADER).read()
    for name, val in (("ULA_ROW_BYTES", 656), ("ULA_ROW_LATENT", 512), ("ULA_ROW_ROPE", 64),
                      ("ULA_ROW_BLOCK", 128), ("ULA_ROPE_PAIRS", ula.ROPE_PAIRS), ("ULA_MAX_AXES", ula.MAX_AXES)):
        m = re.search(rf"#define {name} (\d+)u", src)
        assert m and int(m.group(1)) == val, name
    for name, val in (("ULA_PAIR_ADJACENT", ula.PAIR_ADJACENT), ("ULA_PAIR_HALVES", ula.PAIR_HALVES)):
        assert re.search(rf"{name}\s*=\s*{val}\b", src), name


def test_rotary_layout_matches_header(ula, tmp_path):
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ula.h"\n'
                   "int main(void) { printf(\"%zu %zu %zu %zu %zu\\n\", sizeof(ula_rotary), "
                   "offsetof(ula_rotary, n_axes), offsetof(ula_rotary, pairing), "
                   "offsetof(ula_rotary, freq), offsetof(ula_rotary, axis)); return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)], check=True)
    want = [int(v) for v in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    r = ula.ula_rotary
    assert want == [C.sizeof(r), r.n_axes.offset, r.pairing.offset, r.freq.offset, r.axis.offset]


def test_calls_refuse_null(ula):
    none, u32, u64 = C.c_void_p(), C.c_uint32, C.c_uint64
    lib = ula.lib
    assert lib.ula_rows_attend(none, none) == ula.ERR_INVALID_ARG
    assert lib.ula_rows_rotate(none, u32(0), none, u64(0), u32(1), u32(1), u32(0), none, u64(0), u64(0),
                               none, u64(0), u64(0), none) == ula.ERR_INVALID_ARG
    assert lib.ula_rows_pack(none, none, u64(0), u32(1), u32(0), none, u64(0), none, u64(0), none, u64(656),
                             none) == ula.ERR_INVALID_ARG
    assert lib.ula_rows_join(none, none, u32(1), u64(1), none, none, none) == ula.ERR_INVALID_ARG


def test_rotary_refusals(ula):
    from serving_step_sparse_gb300 import rows
    freq = [1.0] * 32
    assert rows.Rotary(freq).n_axes == 1
    assert rows.Rotary(freq, [0, 1, 2, 0] * 8).n_axes == 3
    for bad in (dict(freq=freq[:31]), dict(freq=freq, axis=[0] * 31), dict(freq=freq, axis=[ula.MAX_AXES] + [0] * 31),
                dict(freq=freq, axis=[-1] + [0] * 31), dict(freq=freq, pairing="thirds")):
        with pytest.raises(ValueError):
            rows.Rotary(**bad)


def test_host_tensors_are_refused(ula):
    from serving_step_sparse_gb300 import rows
    rot = rows.Rotary([1.0 / (j + 1) for j in range(32)])
    pos = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        rows.rotate(torch.zeros(2, 64), pos, rot)
    with pytest.raises(ValueError):
        rows.pack(torch.zeros(2, 512), torch.zeros(2, 64), pos, rot)
    with pytest.raises(ValueError):
        rows.attend(torch.zeros(1, 1, 1, 576, dtype=torch.bfloat16), torch.zeros(4, 656, dtype=torch.uint8),
                    torch.zeros(1, 1, 4, dtype=torch.int32), math.sqrt(1 / 576))
    with pytest.raises(ValueError):
        rows.join([torch.zeros(1, 512, dtype=torch.bfloat16)], [torch.zeros(1)])


def test_rotary_copies_own_their_memory(ula, monkeypatch):
    """A copied or unpickled rotary is read from its own memory, whatever became of the first."""
    import copy
    import gc
    import pickle
    import types
    from serving_step_sparse_gb300 import rows
    freq = [1.0 / (j + 1) for j in range(32)]
    first, second = rows.Rotary(freq, [0, 1] * 16, "halves"), rows.Rotary(freq, [0, 1] * 16, "halves")
    assert pickle.dumps(first) == pickle.dumps(second)      # what it says, not where it stands
    read = []

    def call(x, pos, rotary, *rest):
        read.append(rotary if isinstance(rotary, int) else C.addressof(rotary))

    monkeypatch.setattr(rows, "_rows", types.SimpleNamespace(rotate=call, pack=call))
    for make in (copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r))):
        first = rows.Rotary(freq, [0, 1] * 16, "halves")
        other = make(first)
        del first
        gc.collect()
        rows.rotate(None, None, other)
        assert read[-1] == C.addressof(other.config)
        assert bytes(other.config) == bytes(second.config) and other.n_axes == 2


def test_binding_refuses_a_rotary_of_another_size(ula):
    from serving_step_sparse_gb300 import rows
    for bad in (bytes(8), (C.c_char * 1024)()):
        with pytest.raises(ValueError):
            rows._rows.rotate(torch.zeros(2, 64), torch.zeros(2, dtype=torch.int32), bad, None, False)
    with pytest.raises(TypeError):
        rows._rows.rotate(torch.zeros(2, 64), torch.zeros(2, dtype=torch.int32), 8, None, False)


def test_debug_hold_refuses_other_barriers(ula):
    src = open(HEADER).read()
    n = int(re.search(r"#define ULA_DEBUG_BARRIERS (\d+)", src).group(1))
    try:
        ula.ula_rows_debug_hold(n - 1)
        for bad in (n, 1 << 30):
            with pytest.raises(ula.UlaError) as e:
                ula.ula_rows_debug_hold(bad)
            assert e.value.code == ula.ERR_INVALID_ARG
    finally:
        ula.ula_rows_debug_hold(-1)


def test_sync_is_made_on_the_streams_device(ula, monkeypatch):
    import contextlib
    import types
    from serving_step_sparse_gb300 import rows
    log = []

    @contextlib.contextmanager
    def device(d):
        log.append(("on", d))
        yield
        log.append(("off", d))

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(ula, "ula_rows_sync", lambda s: log.append(("sync", s)))
    rows.sync(types.SimpleNamespace(device="cuda:3", cuda_stream=77))
    assert log == [("on", "cuda:3"), ("sync", 77), ("off", "cuda:3")]


@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls that are let through would launch on no memory")
def test_rotate_refuses_an_output_over_itself(ula):
    """Against every pair of rows, over strides that nest, interleave and collide."""
    import itertools
    rot = ula.ula_rotary()
    rot.n_axes = 1
    u32, u64, at = C.c_uint32, C.c_uint64, C.c_void_p(1 << 20)
    strides = [0, 1, 63, 64, 65, 96, 100, 127, 128, 160, 192, 200, 256, 320, 576]
    for n, heads in ((1, 1), (1, 3), (4, 1), (2, 2), (3, 5), (7, 4)):
        for st, sh in itertools.product(strides, strides):
            starts = sorted(t * st + h * sh for t in range(n) for h in range(heads))
            apart = all(b - a >= 64 for a, b in zip(starts, starts[1:]))
            code = ula.lib.ula_rows_rotate(C.byref(rot), u32(0), at, u64(0), u32(n), u32(heads), u32(0), at, u64(0),
                                           u64(0), at, u64(st), u64(sh), None)
            assert code == (ula.ERR_CUDA if apart else ula.ERR_INVALID_ARG), (n, heads, st, sh)


def test_tensors_that_require_a_gradient_are_refused(ula):
    from serving_step_sparse_gb300 import rows
    rot = rows.Rotary([1.0] * 32)
    pos, x = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 64, requires_grad=True)
    q = torch.zeros(1, 1, 1, 576, dtype=torch.bfloat16, requires_grad=True)
    part = torch.zeros(1, 512, dtype=torch.bfloat16, requires_grad=True)
    calls = [lambda: rows.rotate(x, pos, rot),
             lambda: rows.pack(torch.zeros(2, 512, requires_grad=True), x.detach(), pos, rot),
             lambda: rows.attend(q, torch.zeros(4, 656, dtype=torch.uint8), torch.zeros(1, 1, 4, dtype=torch.int32), 1.0),
             lambda: rows.join([part], [torch.zeros(1)])]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="device"):    # (host tensors)
            call()
