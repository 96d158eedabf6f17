"""The build's commands (no compilation): every HIP source is compiled for
gfx950 with packed fp32 instructions disabled, and only the forward source
gets the memory-clause scheduling strategy."""
import os
import sys

import pytest

from selective_state_space_scan_amd import build as B


def _obj(src):
    return B.object_command("/tmp/x.o", src)


def test_every_source_for_gfx950_without_packed_fp32():
    for src in B.SRCS + [B.PEAKS_SRC]:
        cmd = _obj(src)
        assert "--offload-arch=gfx950" in cmd
        i = cmd.index("-packed-fp32-ops")
        assert cmd[i - 3:i] == ["-Xclang", "-target-feature", "-Xclang"]
        assert "-O3" in cmd and cmd[-4:] == ["-c", src, "-o", "/tmp/x.o"]


def test_scheduling_strategy_only_for_the_forward():
    flag = "-amdgpu-sched-strategy=max-memory-clause"
    fwd = [s for s in B.SRCS if os.path.basename(s) == "ssm_scan.hip"]
    assert len(fwd) == 1 and flag in _obj(fwd[0])
    for src in B.SRCS + [B.PEAKS_SRC]:
        if src not in fwd:
            assert flag not in _obj(src), src


def test_link_command():
    cmd = B.link_command("/tmp/lib.so", ["/tmp/a.o", "/tmp/b.o"])
    assert "-shared" in cmd and "--offload-arch=gfx950" in cmd and cmd[-2:] == ["/tmp/a.o", "/tmp/b.o"]


def _build_with(tmp_path, monkeypatch, run):
    """build() into a folder of its own, its commands given to `run` instead of a compiler."""
    for name in ("LIB_PATH", "PEAKS_LIB_PATH", "TORCH_LIB_PATH"):
        monkeypatch.setattr(B, name, str(tmp_path / os.path.basename(getattr(B, name))))
    done = []

    def fake(cmd, verbose):
        run(cmd)
        done.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(B, "_run", fake)
    return done


def test_libraries_build_without_torch(tmp_path, monkeypatch):
    """A user of the C ABI alone has hipcc and need not have torch: the libraries come out, no module does, and an older
    module, whose structs might not be the library's, does not stay."""
    _build_with(tmp_path, monkeypatch, lambda cmd: None)
    monkeypatch.setitem(sys.modules, "torch", None)   # import torch raises ImportError
    old = tmp_path / os.path.basename(B.TORCH_LIB_PATH)
    old.write_text("older")
    with pytest.warns(RuntimeWarning, match="torch"):
        path = B.build()
    assert path == B.LIB_PATH and os.path.exists(path) and os.path.exists(B.PEAKS_LIB_PATH)
    assert not old.exists()


def test_libraries_build_without_a_host_compiler(tmp_path, monkeypatch):
    def run(cmd):
        if cmd[0] == "g++":
            raise FileNotFoundError("g++")

    _build_with(tmp_path, monkeypatch, run)
    with pytest.warns(RuntimeWarning, match=r"g\+\+"):
        assert os.path.exists(B.build())
    assert not os.path.exists(B.TORCH_LIB_PATH)


def test_a_module_that_does_not_compile_is_an_error_behind_the_libraries(tmp_path, monkeypatch):
    def run(cmd):
        if cmd[0] == "g++":
            raise RuntimeError("g++ failed (1)")

    _build_with(tmp_path, monkeypatch, run)
    with pytest.raises(RuntimeError):
        B.build()
    assert os.path.exists(B.LIB_PATH) and os.path.exists(B.PEAKS_LIB_PATH)
