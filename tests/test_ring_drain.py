"""A kernel that gives up waits for the copies it has in flight before its block ends.  Which barriers those are, and in which
phase, on the host: the function that the kernels use, compiled against barriers that count their phases."""
import os
import re
import subprocess

import pytest

from cross_loop_sparsity_b200 import build as fl_build

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "fl_serving.h"
// A barrier's phase completes when its load arrives; a wait on a parity passes once the current phase has another one.
struct Barrier {
  int phase = 0;
  bool passes(int parity) const { return (phase & 1) != parity; }
};
int main() {
  for (int slots = 1; slots <= 6; ++slots)
    for (long long issued = 0; issued <= 40; ++issued)
      for (long long arrived = issued > slots ? issued - slots : 0; arrived <= issued; ++arrived) {
        std::vector<Barrier> bar(slots);
        for (long long n = 0; n < arrived; ++n) ++bar[n % slots].phase;   // the others are under way
        std::vector<int> asked(slots);
        int blocked = 0;
        fl::each_in_flight(issued, slots, [&](int slot, int parity) {
          ++asked[slot];
          blocked += !bar[slot].passes(parity);
        });
        bool once = true;
        for (int s = 0; s < slots; ++s) once &= asked[s] == (s < issued);
        if (!once || blocked != issued - arrived) {
          std::printf("%d slots, %lld issued, %lld arrived: %d blocked\n", slots, issued, arrived, blocked);
          return 1;
        }
      }
  return 0;
}
"""


def test_every_load_in_flight_is_waited_for(tmp_path):
    src, exe = tmp_path / "drain.cu", tmp_path / "drain"
    src.write_text(PROGRAM)
    subprocess.run([fl_build._nvcc(), "-std=c++17", f"-I{fl_build.INCLUDE}", f"-I{fl_build.CSRC}", "-o", str(exe), str(src)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("kernel,rings", [("k_prefix_split", ["full"]), ("k_prefix_rows", ["full"]),
                                          ("k_prefix_tc", ["k_full", "v_full"]), ("k_weights_stream", ["full"]),
                                          ("k_weights_tc", ["k_full", "q_full"])])
def test_kernels_that_give_up_wait_for_their_rings(kernel, rings):
    """Every ring that a kernel's copies arrive on, by that function."""
    with open(os.path.join(fl_build.CSRC, "fl_prefix.cu")) as f:
        text = f.read()
    at = re.search(r"\n    %s\(|void __launch_bounds__\([^)]*\) %s\(" % (kernel, kernel), text).start()
    body = text[at:text.index("\n}\n", at)]
    waits = re.findall(r"each_in_flight\([^;]*?smem_u32\(&(\w+)\[[^;]*;", body)
    assert sorted(set(waits)) == sorted(rings)
