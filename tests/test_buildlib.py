"""What the build compiles when: the C library needs nvcc alone, the Python binding the torch that it is for.
No compiler runs here."""
import os

import pytest


@pytest.fixture
def build(monkeypatch, tmp_path):
    """buildlib with a folder of its own and compilers that only write their output files; `did` lists them."""
    from gemm_rocmfp2_mul_gb300 import buildlib as b
    for name, value in (("BUILD", tmp_path), ("LIB", tmp_path / "librfp2.so"), ("BINDING", tmp_path / "_rfp2_binding.so")):
        monkeypatch.setattr(b, name, str(value))
    did = []

    def run(cmd, *_, **__):
        out = cmd[cmd.index("-o") + 1]
        what = {"g++": "g++"}.get(cmd[0], "nvcc") + (" link" if "-shared" in cmd else "")
        if what == "g++" and b.broken:
            raise RuntimeError("g++ failed")
        did.append(what)
        open(out, "w").close()
        return ""

    def compile(src):
        obj = os.path.join(b.BUILD, os.path.basename(src)[:-3] + ".o")
        run(["nvcc", "-c", src, "-o", obj])
        return obj, ""

    monkeypatch.setattr(b, "broken", False, raising=False)
    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "_compile", compile)
    monkeypatch.setattr(b, "_nvcc", lambda: "nvcc")
    return b, did


def test_the_library_builds_without_torch(build, monkeypatch):
    import importlib.util
    b, did = build
    monkeypatch.setattr(b, "_torch_dir", lambda: pytest.fail("torch was looked for"))
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert b.build() == b.LIB and os.path.exists(b.LIB) and not os.path.exists(b.BINDING)
    assert did[-1] == "nvcc link" and "g++" not in did
    assert b.up_to_date()


def test_a_binding_that_does_not_compile_leaves_the_library(build, monkeypatch):
    b, did = build
    b.broken = True
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        b.build()
    assert os.path.exists(b.LIB) and did[-1] == "nvcc link"


def test_another_torch_has_the_binding_built_again(build, monkeypatch):
    import importlib.metadata
    b, did = build
    b.build()
    assert did[-2:] == ["nvcc link", "g++ link"] and b.up_to_date()
    did.clear()
    b.build()
    assert not did
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.1" if name == "torch" else version(name))
    assert not b.up_to_date()
    b.build()
    assert did == ["g++", "g++ link"] and b.up_to_date()
