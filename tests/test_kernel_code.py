"""What the compiled kernels rest on, where the language and not a lucky
register allocation has to keep it right."""
import pytest

import kernel_code

pytestmark = pytest.mark.skipif(not kernel_code.available(), reason="needs the ROCm compiler")


@pytest.fixture(scope="module")
def embedding(tmp_path_factory):
    return kernel_code.compile_ir("embedding.hip", tmp_path_factory.mktemp("ir"))


def test_lanes_are_active_where_their_entries_are_read(embedding):
    """Waves over wide rows keep places' entries in the registers of their first
    lanes.  A register of a lane that has left holds nothing for sure (a copy or
    a spill moves the active lanes alone), so every such read stands where no
    lane has left, also at a row's last, partly filled 256 columns."""
    kernels = kernel_code.functions(embedding, ("wide_places_kernel", "wide_table_kernel"))
    assert len(kernels) == 8                       # two kernels, two types, padding or none
    for name, blocks in kernels.items():
        apart, reads = kernel_code.parted(blocks), 0
        for label, block in blocks.items():
            n = sum("llvm.amdgcn.readlane" in line for line in block.lines)
            reads += n
            assert n == 0 or label not in apart, f"{name}: block {label}"
        assert reads > 0, name


@pytest.fixture(scope="module")
def linear_grad(tmp_path_factory):
    return kernel_code.compile_ir("linear_grad.hip", tmp_path_factory.mktemp("ir"))


def test_lanes_exchange_sums_through_lds_in_order(linear_grad):
    """The weight gradient's sums change lanes through LDS, as binary32 values.
    On every path something orders a lane's write before another lane's read,
    and that read before the next write: a fence (with or without a barrier)."""
    kernels = kernel_code.instructions(linear_grad, ("grad_kernel",))
    assert len(kernels) == 4                       # two tiles, transposed or not
    for name, blocks in kernels.items():
        before = {label: set() for label in blocks}
        todo, writes, reads = list(blocks), 0, 0
        while todo:
            label = todo.pop(0)
            open_ = set(before[label])             # accesses that nothing was put behind yet
            for line in blocks[label].lines:
                if line.startswith("fence "):
                    open_ = set()
                elif line.startswith("store float") and "addrspace(3)" in line:
                    assert "read" not in open_, f"{name}: block {label}: {line}"
                    open_.add("write")
                    writes += 1
                elif " = load " in line and "float" in line and "addrspace(3)" in line:
                    assert "write" not in open_, f"{name}: block {label}: {line}"
                    open_.add("read")
                    reads += 1
            for s in blocks[label].next:
                if not open_ <= before[s]:
                    before[s] |= open_
                    todo.append(s)
        assert writes > 0 and reads > 0, name


def test_a_rows_root_mean_square_is_read_at_any_address(tmp_path):
    """A load that states an alignment of four bytes may become a scalar load
    where a row's threads all read the same value, and those ignore the
    address's last two bits."""
    kernels = kernel_code.instructions(kernel_code.compile_ir("rms_norm.hip", tmp_path),
                                       ("norm_grad_kernel",))
    assert len(kernels) == 22                      # eleven widths, padding or none
    for name, blocks in kernels.items():
        loads = [line for b in blocks.values() for line in b.lines
                 if "load float, ptr addrspace(1)" in line]
        assert loads and all("align 1" in line for line in loads), name
