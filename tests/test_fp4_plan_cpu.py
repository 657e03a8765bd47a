"""How a 4-bit product is cut (csrc/fp4_plan.h, plain host code): an accumulator that shares TMEM columns with the
other one is given back only when all of these are read."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "block_diffusion_speculative_hidden_gb300", "csrc")
FIELDS = ("bn", "m_tiles", "split", "stages", "smem", "second", "shared_last", "shared_first", "sc_first", "cols", "x_tiles",
          "blocks", "grid", "pair")
SOURCE = """
#include "fp4_plan.h"
extern "C" void plan(int nv, int M, int N, int kt, int sms, int size, int* out) {
  const auto c = dflash::fp4_plan(nv != 0, M, N, kt, sms, size, [&](int n) { return sms / n; });
  const int v[] = {%s};
  for (unsigned i = 0; i < sizeof(v) / sizeof(*v); ++i) out[i] = v[i];
}
""" % ", ".join(f"static_cast<int>(c.{f})" for f in FIELDS)


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(SOURCE)
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(at / "plan.cpp"),
                    "-o", str(at / "plan.so")], check=True)
    f = ctypes.CDLL(str(at / "plan.so")).plan

    def call(nv, M, N, kt, size, sms=152):
        out = (ctypes.c_int * len(FIELDS))()
        f(nv, M, N, kt, sms, size, out)
        return dict(zip(FIELDS, out))
    return call


def _read_when_given(c, down, last):
    """Columns of an accumulator that are in registers when the last of its warps gives it back: a warp of either turn
    reads two of its blocks (every other one) and then gives, if none of the `last` first ones is left to it."""
    blocks = -(-c["bn"] // 32)
    read = set()
    for turn in (0, 1):
        for i in range(turn, blocks, 4):
            for j in (i, i + 2):
                if j < blocks:
                    b = blocks - 1 - j if down else j
                    read |= set(range(32 * b, min(32 * b + 32, c["bn"])))
            if i + 4 >= last:
                break
    return read


@pytest.mark.parametrize("nv", [0, 1])
@pytest.mark.parametrize("size", [2, 4])
def test_shared_columns_are_read_before_they_are_given_back(plan, nv, size):
    shared = 0
    for M in [*range(1, 560), 1000, 2176, 8192]:
        for N in (257, 5120, 32768, 50000, 128256, 152064):
            for kt in (1, 4, 16, 24):
                c = plan(nv, M, N, kt, size)
                if c["shared_first"] == 0:
                    assert c["shared_last"] == 0
                    # (one tile a CTA, or two accumulators beside each other)
                    assert c["second"] == 0 or c["second"] >= c["bn"]
                    continue
                shared += 1
                bn, second = c["bn"], c["second"]
                assert 0 < second < bn and c["sc_first"] == second + bn
                assert set(range(second, bn)) <= _read_when_given(c, True, c["shared_last"]), (M, N, kt, c)
                assert set(range(bn - second)) <= _read_when_given(c, False, c["shared_first"]), (M, N, kt, c)
    assert shared > 50 or not nv
