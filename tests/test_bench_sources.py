"""The traffic record's key covers everything the step kernel is compiled from (no GPU)."""
from __future__ import annotations

import os
import shutil
import subprocess

import bench
from persistent_moe_decode_gb300 import build

CSRC = os.path.join(bench.ROOT, "persistent_moe_decode_gb300", "csrc")


def test_the_sources_are_those_the_compiler_names():
    """nvcc's own dependency list of the two units, as far as it lies in the folder."""
    nvcc = os.path.join(build._cuda_home(), "bin", "nvcc")
    seen = set()
    for unit in ("mk_kernel.cu", "mk_kernel_q4.cu"):
        r = subprocess.run([nvcc, "-MM", "-std=c++17", f"-I{build.INCLUDE}", os.path.join(CSRC, unit)], capture_output=True,
                           text=True, check=True)
        deps = r.stdout.replace("\\\n", " ").split(":", 1)[1].split()
        seen |= {os.path.relpath(os.path.realpath(d), os.path.realpath(CSRC)) for d in deps
                 if os.path.realpath(d).startswith(os.path.realpath(bench.ROOT))}
    assert sorted(seen) == bench.step_sources(CSRC)


def test_a_new_header_changes_the_key(tmp_path, monkeypatch):
    copy = tmp_path / "persistent_moe_decode_gb300" / "csrc"
    shutil.copytree(CSRC, copy)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    first = bench.kernel_sha()
    (copy / "mk_other.cuh").write_text("#pragma once\nint a;\n")
    assert bench.kernel_sha() == first                   # not included: not compiled
    layout = copy / "mk_layout.h"
    layout.write_text(layout.read_text() + '// #include "mk_gone.cuh"\n')
    assert bench.kernel_sha() == first
    layout.write_text(layout.read_text() + '#include "mk_other.cuh"\n')
    second = bench.kernel_sha()
    (copy / "mk_other.cuh").write_text("#pragma once\nint b;\n")
    assert len({first, second, bench.kernel_sha()}) == 3
