"""The micro-batch operators on the GPU at the edges of their kernels: last,
partly filled groups of columns, turns of a block, addresses, calls at the same
time."""
import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_step_amd as z
from micrograd_ref import Flat, f64, layout
from test_gpu_micrograd import BF16, DEV, emb_exact, some_ids

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free_gpu_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def small_ints(seed, *shape, dtype=BF16):
    return torch.from_numpy(np.random.default_rng(seed).integers(-4, 5, shape)).to(dtype).to(DEV)


@pytest.mark.parametrize("gaps", [False, True])
@pytest.mark.parametrize("flags", [0, z.ACC_OVERWRITE, z.ACC_EMIT_BF16])
@pytest.mark.parametrize("cols", [125, 128, 253, 256, 257, 260, 261, 509, 513, 772])
def test_emb_grad_of_rows_that_leave_lanes_without_columns(cols, flags, gaps):
    """A wave takes 256 columns; the last one of a row as few as one.  Ids of
    one token, of several pieces and of 1024 tokens and more; sums of small
    integers, exact in any order."""
    vocab, n = 90, 2600
    ids = some_ids("uniform", n, vocab, cols)
    ids[100:1300] = 7
    ids[1300:1320] = 8
    ids[::13] = -1
    L, pl = layout(vocab * cols, gaps)
    dy = small_ints(cols, n, cols)
    f = Flat(L, pl, vocab * cols, DEV, ints=True)
    z.zero_embedding_grad(L, 1, torch.from_numpy(ids).to(DEV), dy, f.acc, 1.0, flags, f.out)
    g, _ = emb_exact(ids, f64(dy), vocab)
    want = (0 if flags & z.ACC_OVERWRITE else f.acc0[f.pos]) + g
    assert np.array_equal(f64(f.acc)[f.pos], want)
    f.check(g, np.zeros(g.size), 1.0, flags, f"{cols}")
