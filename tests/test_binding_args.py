"""_args.so, the native check of tensors, is needed by the calls that use it and by nothing else (no GPU needed)."""

import os
import subprocess
import sys

import pytest

from moe_grouped_matmul_amd import build, dg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import sys
sys.modules["moe_grouped_matmul_amd._args"] = None  # importing it fails
import torch
from moe_grouped_matmul_amd import dg
lib = dg.load_library()
assert dg.dg_version() and dg.dg_get_m_alignment_for_contiguous_layout() == 128
assert lib.dg_fp8_gemm_nt(0x10000, 0x10000, 0x10000, 0x10000, 0x10000, 4, 16, 100, None, 0, None) == dg.DG_ERR_SHAPE
assert dg.dg_get_workspace_size(dg.DG_OP_MOE_GATE, 700, 64, 4) > 0
for _ in range(2):
    try:
        dg._arg(torch.zeros(2, 3), "x", torch.float32, (2, 3), 0)
    except RuntimeError as e:
        assert "_args.so" in str(e) and isinstance(e.__cause__, ImportError)
    else:
        raise AssertionError("no error")
print("done")
"""


def test_library_loads_without_it():
    if not os.path.exists(dg.LIB_PATH):
        build.build()
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("done"), r.stderr[-2000:]


def test_library_builds_without_it(monkeypatch, tmp_path, capsys):
    src = tmp_path / "part.c"
    src.write_text("int part(void) { return 7; }\n")

    def compile_part(name, build_dir, extra):
        obj = os.path.join(build_dir, name + ".o")
        subprocess.run(["gcc", "-fPIC", "-c", str(src), "-o", obj], check=True)
        return obj, ""

    def no_compiler():
        raise RuntimeError("no g++")

    lib, args = tmp_path / "lib.so", tmp_path / "_args.so"
    args.write_text("older")
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "b"))
    monkeypatch.setattr(build, "LIB_PATH", str(lib))
    monkeypatch.setattr(build, "ARGS_PATH", str(args))
    monkeypatch.setattr(build, "SOURCES", ["part"])
    monkeypatch.setattr(build, "_compile", compile_part)
    monkeypatch.setattr(build, "_build_args", no_compiler)
    assert build.build() == str(lib) and lib.exists()
    assert not args.exists() and "no g++" in capsys.readouterr().err


def test_library_errors_still_end_the_build(monkeypatch, tmp_path):
    def fails(name, build_dir, extra):
        raise RuntimeError("hipcc failed")

    monkeypatch.setattr(build, "BUILD", str(tmp_path / "b"))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "ARGS_PATH", str(tmp_path / "_args.so"))
    monkeypatch.setattr(build, "_compile", fails)
    monkeypatch.setattr(build, "_build_args", lambda: None)
    with pytest.raises(RuntimeError, match="hipcc failed"):
        build.build()
