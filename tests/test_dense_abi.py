"""The cache writer and the dense attention without a GPU: mirrored structs
and refusals on the host, before anything is enqueued."""
import ctypes as C
import os
import shutil
import subprocess

import pytest
import torch

import helpers
from test_abi import _problem

HEADER = os.path.join(helpers.ROOT, "include")
FAKE = 1 << 30


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
@pytest.mark.parametrize("name", ["msa_rope", "msa_append"])
def test_struct_layout_matches_header(tmp_path, name):
    import block_sparse_attention_index_gb300 as m
    mirror = {"msa_rope": m.MsaRope, "msa_append": m.MsaAppend}[name]
    fields = [f for f, _ in mirror._fields_]
    prog = '#include <stdio.h>\n#include <stddef.h>\n#include "msa.h"\nint main(void){\n'
    prog += 'printf("%%zu\\n", sizeof(%s));\n' % name
    prog += "".join('printf("%%zu\\n", offsetof(%s, %s));\n' % (name, f) for f in fields) + "return 0;}\n"
    (tmp_path / "t.c").write_text(prog)
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-I", HEADER, str(tmp_path / "t.c"), "-o", str(exe)], check=True)
    vals = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert vals == [C.sizeof(mirror)] + [getattr(mirror, f).offset for f in fields]


def _append(**over):
    import block_sparse_attention_index_gb300 as m
    vals = dict(k=FAKE, v=FAKE, ik=FAKE, q=FAKE, iq=FAKE, k_stride=512, v_stride=512, ik_stride=256, q_stride=8192,
                iq_stride=256, k_cache=FAKE, v_cache=FAKE, ik_cache=FAKE, q_out=2 * FAKE, iq_out=2 * FAKE)
    vals.update(over)
    return m.MsaAppend(**vals)


@pytest.mark.parametrize("over,status", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(k=FAKE + 8), 1), (dict(k_cache=None), 1), (dict(v_cache=FAKE + 4), 1),
    (dict(k_stride=504), 1), (dict(v_stride=516), 1), (dict(q_stride=8188), 1), (dict(iq_stride=-256), 1),
    (dict(ik=None), 1), (dict(ik_cache=None), 1), (dict(q_out=None), 1), (dict(iq=None), 1), (dict(iq_out=FAKE + 2), 1),
    (dict(q_out=FAKE, q_stride=8200), 1), (dict(k_scale=FAKE), 1), (dict(v_scale=FAKE, k_scale=FAKE), 1),
])
def test_append_arguments_rejected_on_host(over, status):
    import block_sparse_attention_index_gb300 as m
    L = m.lib()
    pb, a, ws = _problem(), _append(**over), C.c_void_p(1 << 20)
    assert L.msa_append_cache(C.byref(pb), C.byref(a), None, ws, 256, None) == status
    assert L.msa_last_error()


def test_append_workspace_and_problem_checks():
    import block_sparse_attention_index_gb300 as m
    L = m.lib()
    pb, a, ws = _problem(), _append(), C.c_void_p(1 << 20)
    assert L.msa_append_cache(C.byref(pb), C.byref(a), None, None, 256, None) == 3
    assert L.msa_append_cache(C.byref(pb), C.byref(a), None, ws, 255, None) == 3
    assert L.msa_append_cache(C.byref(pb), C.byref(a), None, C.c_void_p((1 << 20) + 16), 256, None) == 3
    assert L.msa_append_cache(C.byref(pb), None, None, ws, 256, None) == 1
    assert L.msa_append_cache(C.byref(_problem(num_kv_heads=3)), C.byref(a), None, ws, 256, None) == 2
    # an int8 cache needs both scale arrays
    p8 = _problem(kv_dtype=1, k_scale=2048, v_scale=4096)
    assert L.msa_append_cache(C.byref(p8), C.byref(a), None, ws, 256, None) == 1
    assert L.msa_append_cache(C.byref(p8), C.byref(_append(k_scale=FAKE, v_scale=FAKE + 2)), None, ws, 256, None) == 1


@pytest.mark.parametrize("over,status", [
    (dict(dim=8), 2), (dict(dim=144), 2), (dict(dim=-16), 2), (dict(index_dim=80), 2), (dict(axes=0), 2), (dict(axes=5), 2),
    (dict(interleaved=2), 1), (dict(turns=None), 1), (dict(index_turns=None), 1), (dict(axes=2), 1),
    (dict(axes=2, axis=FAKE), 1), (dict(turns=FAKE + 4), 1), (dict(positions=FAKE + 2), 1),
    (dict(axes=2, axis=FAKE + 1, index_axis=FAKE), 1),
])
def test_rope_rejected_on_host(over, status):
    import block_sparse_attention_index_gb300 as m
    vals = dict(dim=64, index_dim=32, axes=1, interleaved=0, turns=FAKE, index_turns=FAKE)
    vals.update(over)
    pb, a, r = _problem(), _append(), m.MsaRope(**vals)
    assert m.lib().msa_append_cache(C.byref(pb), C.byref(a), C.byref(r), C.c_void_p(1 << 20), 256, None) == status
    assert m.lib().msa_last_error()


def test_dense_arguments_rejected_on_host():
    import block_sparse_attention_index_gb300 as m
    L = m.lib()
    pb, n = _problem(), C.c_size_t(0)
    assert L.msa_dense_workspace_size(C.byref(pb), C.byref(n)) == 0 and n.value >= 256 and n.value % 256 == 0
    assert L.msa_dense_workspace_size(C.byref(pb), None) == 1
    assert L.msa_dense_workspace_size(C.byref(_problem(head_dim=64)), C.byref(n)) == 2
    L.msa_dense_workspace_size(C.byref(pb), C.byref(n))
    f, o, ws = C.c_void_p(FAKE), C.c_void_p(FAKE + (1 << 30)), C.c_void_p(1 << 20)
    bad = C.c_void_p(FAKE + 8)
    for args in ((None, f, f, o), (f, None, f, o), (f, f, bad, o), (f, f, f, bad)):
        assert L.msa_dense_forward(C.byref(pb), *args, ws, n.value, None) == 1
    # out must not touch q: the same, its last value, and one that begins inside it
    values = pb.total_rows * pb.num_kv_heads * pb.group_size * 128
    width = 2 if pb.out_dtype else 4
    for at in (FAKE, FAKE + 2 * values - 16, FAKE - width * values + 16):
        assert L.msa_dense_forward(C.byref(pb), f, f, f, C.c_void_p(at), ws, n.value, None) == 1
        assert b"overlaps" in L.msa_last_error()
    for at in (FAKE + 2 * values, FAKE - width * values):  # beside it: on to the workspace's checks
        assert L.msa_dense_forward(C.byref(pb), f, f, f, C.c_void_p(at), None, n.value, None) == 3
    assert L.msa_dense_forward(C.byref(pb), f, f, f, o, None, n.value, None) == 3
    assert L.msa_dense_forward(C.byref(pb), f, f, f, o, ws, n.value - 1, None) == 3
    assert L.msa_dense_forward(C.byref(pb), f, f, f, o, C.c_void_p((1 << 20) + 128), n.value, None) == 3
    assert L.msa_dense_forward(C.byref(_problem(group_size=17)), f, f, f, o, ws, n.value, None) == 2


def test_rope_tables():
    """turns: theta^(-2j/dim) / 2 pi of a turn, in units of 2^-64: off by the cut to a whole unit (below 2^-64; a
    small frequency is a small integer, so this is not a relative error) and a few double roundings (2^-50)."""
    import math

    import block_sparse_attention_index_gb300 as m
    r = m.Rope(64, 32, theta=1e6, device="cpu")
    for t, n in ((r.turns, 64), (r.index_turns, 32)):
        assert t.dtype == torch.int64 and t.numel() == n // 2
        for j, x in enumerate(t.tolist()):
            f = (x % (1 << 64)) / 2.0 ** 64
            want = 1e6 ** (-2 * j / n) / (2 * math.pi)
            assert abs(f - want) <= 2.0 ** -64 + want * 2.0 ** -50
    with pytest.raises(ValueError):
        m.Rope(64, axes=3, device="cpu")
    with pytest.raises(ValueError):
        m.Rope(64, axes=3, axis=[0] * 31, device="cpu")
