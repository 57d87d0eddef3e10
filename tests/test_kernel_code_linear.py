"""What the linear layer's compiled kernels rest on: LDS that lanes exchange, and
LDS that requests fill."""
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


def test_requests_say_what_they_write(linear):
    """m0, which holds a request's place in LDS, and memory: nothing that the
    compiler keeps there itself, and no LDS access, may be moved across one."""
    for name, blocks in linear.items():
        lines = [line for b in blocks.values() for line in b.lines if "global_load_lds_dwordx4" in line]
        assert lines and all("~{m0}" in line and "~{memory}" in line for line in lines), name


def test_fragments_are_read_behind_a_wait_and_a_barrier(linear):
    """On every path a wave waits for its requests, the waves meet, and only then
    fragments are read or further requests put where others were read: nothing of
    either stands between a wait and its barrier, nor a read behind a barrier
    without a wait."""
    for name, blocks in linear.items():
        seen = set()

        def step(state, line):
            if "s_waitcnt vmcnt" in line:
                return frozenset({"waited"})
            if "@llvm.amdgcn.s.barrier()" in line:
                return frozenset({"met"}) if "waited" in state else frozenset({"closed"})
            if "global_load_lds_dwordx4" in line:
                seen.add("request")
                assert state <= {"met", "begun"}, f"{name}: {line}"
            elif "@llvm.amdgcn.ds.read.tr16" in line or (" = load <8 x bfloat>" in line and "addrspace(3)" in line):
                seen.add("read")
                assert state == {"met"}, f"{name}: {line}"
            return state
        walk(blocks, frozenset({"begun"}), step)
        assert seen == {"request", "read"}, name
