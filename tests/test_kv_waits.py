"""The limits of the paged cache's attention's waits against the longest item that a
call may have (no GPU)."""
from __future__ import annotations

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = r"""
#include <cstdio>
#include "mk_kv_sched.cuh"
int main() {
  using namespace mk;
  // 2900 cycles a key tile, the most that a wide one takes, at 1455 MHz, the clock of long matrix products
  const double item = (double)kKvMaxPages * kKvPage / kTile * 2900 / 1.455;
  // a wait of one item's length has room for a clock of a tenth of that, and ends within two minutes
  std::printf("%d\n", 10 * item < (double)kKvItemWaits * kKvWaitNs && (double)kKvItemWaits * kKvWaitNs <= 120e9);
}
"""


def test_no_item_outlasts_the_waits_for_it(tmp_path):
    (tmp_path / "w.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "persistent_moe_decode_gb300", "csrc"), str(tmp_path / "w.cpp"), "-o",
                    str(tmp_path / "w")], check=True)
    assert subprocess.run([str(tmp_path / "w")], capture_output=True, text=True, check=True).stdout == "1\n"
