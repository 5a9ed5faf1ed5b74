"""CPU test of the choice of a cluster size (csrc/cluster_choice.h): sizes that the
device cannot run are passed over, and each size is asked for once."""
import ctypes
import subprocess
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parent.parent / "speculative_decoding_rejection_gb300" / "csrc"
PROGRAM = """
#include "cluster_choice.h"
static std::atomic<int> counts[9];
extern "C" void reset() { for (auto &c : counts) c = 0; }
// has[C]: clusters of C that run, 0 or less: the size does not; asked[C] counts the questions
extern "C" int choose(int least, const int *has, int *asked, int *count) {
  const sv::ClusterChoice c = sv::choose_cluster(
      counts, 8, [&](int C) { return C >= least; }, [&](int C) { ++asked[C]; return has[C]; });
  *count = c.count;
  return c.size;
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    d = tmp_path_factory.mktemp("cluster")
    (d / "c.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{CSRC}", str(d / "c.cpp"), "-o",
                    str(d / "c.so")], check=True)
    L = ctypes.CDLL(str(d / "c.so"))

    def run(least, has, asked=None):
        asked = asked if asked is not None else (ctypes.c_int * 9)()
        n = ctypes.c_int(-5)
        size = L.choose(least, (ctypes.c_int * 9)(0, *has), asked, ctypes.byref(n))
        return size, n.value, list(asked)

    return L, run


@pytest.mark.parametrize("least,has,want", [
    (1, [152, 76, 50, 38, 30, 25, 21, 19], (1, 152)),
    (2, [152, 74, 50, 36, 30, 24, 21, 17], (3, 50)),   # 2: 148 SMs, 3 and 5: 150
    (2, [152, 74, 48, 36, 0, -1, 0, 0], (2, 74)),      # 5 to 8 do not run here
    (5, [152, 74, 48, 36, 0, 0, 0, 0], (0, 0)),        # none that fits does
    (1, [0] * 8, (0, 0)),
])
def test_choice(choose, least, has, want):
    L, run = choose
    L.reset()
    size, count, asked = run(least, has)
    assert (size, count) == want
    assert asked[least:] == [1] * (9 - least) and not any(asked[:least])
    again = (ctypes.c_int * 9)()
    assert run(least, has, again)[:2] == want and not any(again)
