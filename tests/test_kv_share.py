"""The paged cache's attention's shares by the kernel's own formula, on the host
under the address and undefined-behaviour sanitizers (no GPU)."""
from __future__ import annotations

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def checker(tmp_path_factory):
    exe = tmp_path_factory.mktemp("kv_share") / "check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "persistent_moe_decode_gb300", "csrc"), "-x", "c++",
                    os.path.join(ROOT, "tests", "kv_share.cpp"), "-o", str(exe)], check=True)
    return exe


@pytest.mark.parametrize("seed", range(3))
def test_the_blocks_shares_cover_everything_once(checker, seed):
    r = subprocess.run([str(checker), str(seed)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr[-3000:]
