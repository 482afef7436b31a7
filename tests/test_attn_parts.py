"""How an attention call's work is divided among workgroups, by the host's
compiler from the header that the kernels use."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "speculative_decode_verify_gdn_amd", "csrc")
SOURCE = """
#include "attn_parts.hpp"
extern "C" int active(long long total, int n_wg, long long grain, int heads, int idle) {
  return gdn::attn_active(total, n_wg, grain, heads, idle);
}
extern "C" int spread(int block, int active, int xcds) {
  return gdn::attn_spread(block, active, xcds);
}
"""


@pytest.fixture(scope="module")
def parts(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("parts")
    (d / "parts.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC,
                    str(d / "parts.cpp"), "-o", str(d / "parts.so")], check=True)
    lib = ctypes.CDLL(str(d / "parts.so"))
    lib.active.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    return lib


@pytest.mark.parametrize("n_wg", [256, 512])
def test_active_workgroups_are_even_over_the_xcds(parts, n_wg):
    """Every number of the line once; of the active ones each XCD (block modulo 8) has
    the same count to within one, and they are neighbours."""
    for active in range(n_wg + 1):
        wg = np.array([parts.spread(b, active, 8) for b in range(n_wg)])
        assert sorted(wg) == list(range(n_wg)), active
        count = []
        for x in range(8):
            mine = np.sort(wg[x::8][wg[x::8] < active])
            count.append(len(mine))
            assert len(mine) < 2 or (np.diff(mine) == 1).all(), (active, x)
        assert max(count) - min(count) <= 1, (active, count)


@pytest.mark.parametrize("n_wg,grain", [(256, 128), (512, 128), (512, 256), (512, 64)])
def test_active_workgroups(parts, n_wg, grain):
    """Enough for the work, no more than there are, whole heads where that leaves no
    more than `idle` without work."""
    rng = np.random.default_rng(n_wg + grain)
    for _ in range(3000):
        heads, idle = int(rng.integers(1, 700)), int(rng.choice([0, n_wg // 4, n_wg]))
        total = int(np.exp(rng.uniform(0, np.log(1e12))))
        n = parts.active(total, n_wg, grain, heads, idle)
        wanted = min(n_wg, -(-total // grain))
        assert wanted - idle <= n <= n_wg and n >= 1
        if heads <= n_wg and (idle == n_wg or -(-wanted // heads) * heads <= n_wg):
            assert n % heads == 0
        else:
            assert n == wanted or (n % heads == 0 and n_wg - n <= idle)
    assert parts.active(0, n_wg, grain, 4, 0) == 0
