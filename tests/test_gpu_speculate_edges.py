"""The operators of a speculative step at the edges of what their documentation allows."""
import pytest
import torch

import exact_top_selection_amd as ets
from tests import speculate_reference as spec
from tests.test_gpu_speculate import filled, ints
from tests.test_gpu_step import BF16, FP16, FP32, dev, gen

pytestmark = pytest.mark.gpu


# ---- sequences that a write leaves alone

@pytest.mark.parametrize("dtype,D,block", [(BF16, 64, 8), (FP16, 128, 16), (FP32, 256, 40)])  # one wave, and four
def test_block_write_of_no_rows_writes_nothing(dtype, D, block):
    """A sequence with no rows keeps its bytes, whatever they are, though its next position stands inside a block."""
    g = gen(71)
    codes = torch.randint(0, 256, (6 * block, 2, D), generator=g, dtype=torch.uint8)
    scales = torch.tensor([0, 255, 0, 247, 0, 90], dtype=torch.uint8).view(6, 1).repeat(1, 2)
    x = torch.randn(6, block, 2, D, generator=g).to(dtype)
    table = torch.arange(6, dtype=torch.int32).view(6, 1)
    first = ints(2, block - 1, 3, block - 1, -1, 3)
    counts = ints(0, 0, -1, -0x80000000, 4, 0)
    got = codes.to(dev()), scales.to(dev())
    ets.block_write(x.to(dev()), *got, table.to(dev()), first.to(dev()), counts.to(dev()), block)
    assert torch.equal(got[1].cpu(), scales) and torch.equal(got[0].cpu(), codes)
    # next to one that is written
    counts[5] = 2
    scales[5] = 127
    want = spec.block_write(x, codes, scales, table, first, counts, block)
    got = codes.to(dev()), scales.to(dev())
    ets.block_write(x.to(dev()), *got, table.to(dev()), first.to(dev()), counts.to(dev()), block)
    assert torch.equal(got[1].cpu(), want[1]) and torch.equal(got[0].cpu()[:5 * block], codes[:5 * block])
