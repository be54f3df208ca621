"""The layout check of the contiguous forms (DG_CHECK_LAYOUT) reads m_indices a run at a time and allocates nothing that could
throw through the C entries: driven on host memory with allocations refused (tests/host/layout_check.cpp), no GPU needed."""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_layout_check_without_memory(tmp_path):
    from moe_grouped_matmul_amd import build

    objs = [os.path.join(build.BUILD, os.path.splitext(s)[0] + ".o") for s in build.SOURCES]
    if not all(os.path.exists(o) for o in objs):
        build.build()
    inc = ["-I", os.path.join(ROOT, "include"), "-I", build.CSRC, "-I", "/opt/rocm/include"]
    exe = str(tmp_path / "layout_check")
    cmd = ["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", *inc, os.path.join(ROOT, "tests", "host", "layout_check.cpp"), *objs,
           "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "0 failures" in r.stdout, (r.returncode, r.stdout[-2000:], r.stderr[-2000:])
