"""Starts out of order, as the paged cache's attention takes them on the device, on
the host under the address and undefined-behaviour sanitizers (no GPU)."""
from __future__ import annotations

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def checker(tmp_path_factory):
    exe = tmp_path_factory.mktemp("kv_starts") / "check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "persistent_moe_decode_gb300", "csrc"), "-x", "c++",
                    os.path.join(ROOT, "tests", "kv_starts.cpp"), "-o", str(exe)], check=True)
    return exe


@pytest.mark.parametrize("seed", range(4))
def test_rows_have_one_sequence_and_one_group(checker, seed):
    r = subprocess.run([str(checker), str(seed)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr[-3000:]
