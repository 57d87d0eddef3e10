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
