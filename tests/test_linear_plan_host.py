"""The tiles that a product of the linear layer is cut into, without a GPU."""
import ctypes as C
import subprocess

import pytest

import fsdp_sharded_optimizer_step_amd as z
from fsdp_sharded_optimizer_step_amd import build_ext
from linear_cases import LARGE_TILES

DRIVER = """
#include "linear_plan.hpp"
extern "C" void plan(int64_t M, int64_t N, int64_t K, int64_t* tiles, double* us) {
  const zs::TilePlan p = zs::plan_of(M, N, K);
  tiles[0] = p.side, tiles[1] = p.whole, tiles[2] = p.further, tiles[3] = p.splits;
  us[0] = zs::plan_for<4>(M, N, K).us, us[1] = zs::plan_for<2>(M, N, K).us;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    folder = tmp_path_factory.mktemp("plan")
    src, out = str(folder / "plan.cpp"), str(folder / "plan.so")
    with open(src, "w") as f:
        f.write(DRIVER)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I", build_ext.CSRC, src, "-o", out],
                   check=True)
    lib = C.CDLL(out)

    def call(M, N, K):
        tiles, us = (C.c_int64 * 4)(), (C.c_double * 2)()
        lib.plan(C.c_int64(M), C.c_int64(N), C.c_int64(K), tiles, us)
        return tuple(tiles), tuple(us)
    return call


def at(n):
    """A host address standing in for a device pointer; never read."""
    return C.c_void_p(0x10000000 * n)


@pytest.mark.parametrize("size", LARGE_TILES)
def test_large_tiles_are_chosen(plan, size):
    """With a margin in the estimate, so that a change of its figures shows here
    before these sizes stop running the larger tile's kernels."""
    (side, whole, further, splits), (large, small) = plan(*size)
    assert side == 256 and small > 1.04 * large
    assert ("whole" in LARGE_TILES[size]) == (whole > 0)
    assert ("split" in LARGE_TILES[size]) == (further > 0) and (splits > 1) == (further > 0)


@pytest.mark.parametrize("tr", [0, 1])
@pytest.mark.parametrize("size", [s for s in LARGE_TILES if LARGE_TILES[s][-1] == "split"])
def test_the_library_cuts_products_so(plan, size, tr):
    """The workspace is the split tiles' parts, beside the copies of what has no
    whole chunks."""
    lib, (M, N, K) = z.load(), size
    (side, _, further, splits), _ = plan(*size)
    whole = lambda n: (n + 7) // 8 * 8  # noqa: E731
    L = z.Layout([16, N * K], 0, 4, 1)
    for grad in (False, True):
        f = lib.zero_linear_input_grad_workspace if grad else lib.zero_linear_workspace
        o, i = (K, N) if grad else (N, K)
        rows, cols = (i, o) if tr else (o, i)
        copies = (2 * rows * whole(cols) if cols % 8 else 0) + (2 * M * whole(K) if K % 8 else 0)
        assert f(L.handle, 1, tr, at(1), at(2), K, M, o, i) == copies + further * splits * side * side * 4
