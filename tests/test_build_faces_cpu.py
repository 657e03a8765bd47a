"""The compiled faces are rebuilt when they meet another PyTorch or Python, however old its files are."""
import os
import sys


def test_another_pytorch_is_a_reason_to_compile(tmp_path, monkeypatch):
    from block_diffusion_speculative_hidden_gb300 import build_lib
    runs = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("object")
        return Done
    monkeypatch.setattr(build_lib, "BUILD", str(tmp_path / "out"))
    os.makedirs(build_lib.BUILD)
    monkeypatch.setattr(build_lib.subprocess, "run", run)

    def torch_at(name, version):
        d = tmp_path / name
        d.mkdir(exist_ok=True)
        (d / "version.py").write_text(f"__version__ = '{version}'\n")
        os.utime(d / "version.py", (1, 1))           # far older than any object
        monkeypatch.setattr(build_lib, "_torch_dir", lambda: str(d))

    def compiled():
        n = len(runs)
        obj = build_lib._compile_faces()
        assert os.path.exists(obj)
        return len(runs) - n
    torch_at("torch", "2.11.0")
    assert compiled() == 1 and compiled() == 0
    torch_at("torch", "2.9.1")                       # the same place
    assert compiled() == 1 and compiled() == 0
    torch_at("elsewhere", "2.9.1")                   # the same version
    assert compiled() == 1 and compiled() == 0
    monkeypatch.setattr(sys, "version", "3.13.0")
    assert compiled() == 1 and compiled() == 0
    os.remove(os.path.join(build_lib.BUILD, "faces.o"))
    assert compiled() == 1 and compiled() == 0


def test_a_failed_compile_is_tried_again(tmp_path, monkeypatch):
    import pytest
    from block_diffusion_speculative_hidden_gb300 import build_lib
    runs = []

    class Failed:
        returncode, stdout, stderr = 1, "", "no header"

    monkeypatch.setattr(build_lib, "BUILD", str(tmp_path))
    monkeypatch.setattr(build_lib.subprocess, "run", lambda cmd, **kw: runs.append(cmd) or Failed)
    for n in (1, 2):
        with pytest.raises(RuntimeError, match="no header"):
            build_lib._compile_faces()
        assert len(runs) == n
