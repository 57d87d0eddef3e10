"""What the linear layer's compiled kernels rest on: LDS that lanes exchange."""
import pytest

import kernel_code

pytestmark = pytest.mark.skipif(not kernel_code.available(), reason="needs the ROCm compiler")


@pytest.fixture(scope="module")
def linear(tmp_path_factory):
    ir = kernel_code.compile_ir("linear.hip", tmp_path_factory.mktemp("ir"))
    kernels = kernel_code.instructions(ir, ("product_kernel",))
    assert len(kernels) == 4                       # two tiles, two orders of the weight
    return kernels


def walk(blocks, start, step):
    """Facts (frozensets) that hold on some path into each block, to a fixed
    point; step(facts, line) -> facts."""
    before = {label: set() for label in blocks}
    before[""] = {start}
    todo = [""]
    while todo:
        label = todo.pop(0)
        for facts in list(before[label]):
            for line in blocks[label].lines:
                facts = step(facts, line)
            for s in blocks[label].next:
                if facts not in before[s]:
                    before[s].add(facts)
                    todo.append(s)
    return before


def test_lanes_exchange_sums_through_lds_in_order(linear):
    """A wave's sums change lanes through LDS as binary32 values: on every path a
    fence stands between a lane's write and another lane's read, and between that
    read and the next write."""
    for name, blocks in linear.items():
        seen = set()

        def step(open_, line):
            if line.startswith("fence "):
                return frozenset()
            if line.startswith("store <4 x float>") and "addrspace(3)" in line:
                assert "read" not in open_, f"{name}: {line}"
                seen.add("write")
                return open_ | {"write"}
            if " = load <4 x float>" in line and "addrspace(3)" in line:
                assert "write" not in open_, f"{name}: {line}"
                seen.add("read")
                return open_ | {"read"}
            return open_
        walk(blocks, frozenset(), step)
        assert seen == {"write", "read"}, name
