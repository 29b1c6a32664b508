"""Idle slots of a padded batch, as the paged cache's attention walks past them, on
the host under the address sanitizer (no GPU)."""
from __future__ import annotations

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_stretch_ends_before_the_idle_slots_behind_it(tmp_path):
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-Wall", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "persistent_moe_decode_gb300", "csrc"), "-x", "c++",
                    os.path.join(ROOT, "tests", "kv_idle.cpp"), "-o", str(tmp_path / "idle")], check=True)
    r = subprocess.run([str(tmp_path / "idle")], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr[-3000:]
