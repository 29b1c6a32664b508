"""The shares that the paged cache's attention cuts on the device, walked on the
host under the address and undefined-behaviour sanitizers (no GPU)."""
from __future__ import annotations

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def walker(tmp_path_factory):
    exe = tmp_path_factory.mktemp("kv_sched") / "walk"
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "persistent_moe_decode_gb300", "csrc"), "-x", "c++",
                    os.path.join(ROOT, "tests", "kv_sched.cpp"), "-o", str(exe)], check=True)
    return exe


@pytest.mark.parametrize("seed", range(4))
def test_every_tile_is_taken_once(walker, seed):
    r = subprocess.run([str(walker), "250", str(seed)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr[-3000:]
