"""CPU: the binding's native half is needed by the calls that go through it and by nothing else. The library
builds without it, the other entry points load without it, and one built for another interpreter or torch is
rebuilt, and not loaded meanwhile."""
import os
import subprocess
import sys
import warnings

import pytest

from differential_attention_v2_b200 import build as b

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_library_is_built_where_the_native_half_cannot_be(monkeypatch):
    made = []
    monkeypatch.setattr(b, "_compile", lambda out, *a: made.append(out))

    def missing(**kw):
        assert made  # the library comes first
        raise ImportError("no torch here")

    monkeypatch.setattr(b, "build_native", missing)
    with pytest.warns(UserWarning, match="no torch here"):
        assert b.build(force=True) == b.LIB_PATH
    assert made == [b.LIB_PATH]
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        b.build(force=True, debug_bounds=True)


def test_one_built_for_another_torch_is_rebuilt(tmp_path, monkeypatch):
    so, stamp = tmp_path / "_native.so", tmp_path / "_native.stamp"
    monkeypatch.setattr(b, "NATIVE_PATH", str(so))
    monkeypatch.setattr(b, "NATIVE_STAMP_PATH", str(stamp))
    runs = []

    def compiler(cmd, **kw):
        runs.append(cmd)
        with open(str(so) + ".tmp", "w") as f:
            f.write("new")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", compiler)
    for said, rebuilt in ((None, True), ("python cpython-311 torch 1.0", True), (b.native_stamp(), False)):
        so.write_text("old")
        stamp.unlink(missing_ok=True)
        if said is not None:
            stamp.write_text(said)
        b.build_native()
        assert so.read_text() == ("new" if rebuilt else "old") and stamp.read_text() == b.native_stamp()
    assert len(runs) == 2


LOADS = """
import sys
from differential_attention_v2_b200 import build
build.NATIVE_PATH, build.NATIVE_STAMP_PATH = sys.argv[1:]
import differential_attention_v2_b200 as da
assert da.version() >= 100 and da.decode_workspace_size(1, 4096, 8, 2, 128) > 0
import torch
t = torch.zeros(1)
try:
    da.prefill(t, t, t, t)
except (TypeError, ValueError):  # the call's own checks: a CPU tensor
    pass
for call in (lambda: da.rope(t, None, t, t, (1,)), lambda: da.decode(t, t, t, t, t, window=1, sink=1),
             lambda: da.cache_trim(t, t, t, 8, 1, 1)):
    try:
        call()
    except ImportError as e:
        print(e)
"""


@pytest.mark.parametrize("case", ["missing", "other torch", "unloadable"])
def test_the_other_entry_points_load_without_it(tmp_path, case):
    b.build()
    so, stamp = tmp_path / "_native.so", tmp_path / "_native.stamp"
    if case != "missing":
        so.write_text("not a shared object")
    if case == "other torch":
        stamp.write_text("python cpython-311 torch 1.0")
    out = subprocess.run([sys.executable, "-c", LOADS, str(so), str(stamp)], cwd=ROOT, capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    lines = out.stdout.splitlines()
    assert len(lines) == 3 and all("differential_attention_v2_b200.build" in x for x in lines), out.stdout


ROPE = """q:io<T,Hq,D> k:io<T,Hkv,D>? positions:i32[%.n,T] inv_freq:f32[%.sum] %sections
    >q_out:io<T,Hq,D> >k_out:io<T,Hkv,D>?k !inverse !interleaved
    -> q k q_out k_out positions inv_freq % %.n T Hq Hkv D q.s k.s q_out.s k_out.s io interleaved inverse => q_out"""
SIZED = """q:bf16[B,S,Hq,D] k:bf16[B,S,Hkv,D] v:bf16[B,S,Hkv,D] lam:f32[B,S,Hq/2] o_branch:f32[B,S,Hq,D]
    lse:f32[B,S,Hq] dout:bf16[B,S,Hq/2,D] #window #sink >dq:bf16[B,S,Hq,D] >dk:bf16[B,S,Hkv,D] >dv:bf16[B,S,Hkv,D]
    >dlam:f32[B,S,Hq/2] @workspace(B,S,Hq,Hkv,window,sink)
    -> q k v lam o_branch lse dout dq dk dv dlam B S Hq Hkv D window sink workspace workspace.n => dq"""


def test_a_description_that_does_not_fit_its_prototype_is_refused():
    from differential_attention_v2_b200 import _lib

    _lib._check_description("diffattn_v2_rope", ROPE)
    _lib._check_description("diffattn_v2_backward_window_sink", SIZED)
    for name, right, a, b in (("rope", ROPE, " k.s", ""), ("rope", ROPE, " inverse =>", " inverse D =>"),
                              ("rope", ROPE, "T Hq Hkv D q.s", "q Hq Hkv D q.s"), ("rope", ROPE, "% %.n", "%.n %"),
                              ("backward_window_sink", SIZED, "(B,S,", "(S,"),
                              ("backward_window_sink", SIZED, "workspace workspace.n", "workspace")):
        assert a in right
        with pytest.raises(TypeError):
            _lib._check_description("diffattn_v2_" + name, right.replace(a, b))
