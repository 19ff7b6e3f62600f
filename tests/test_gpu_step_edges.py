"""The decode operators where their arithmetic or their lists come to an edge, against tests/decode_reference.py."""
import math

import pytest
import torch

import exact_top_selection_amd as ets
from tests import decode_reference as ref
from tests.test_gpu_step import BF16, FP16, FP32, attention_case, cache, close, dev, gen

pytestmark = pytest.mark.gpu


def two_parts(q, *args):
    """ref.attend with the bound of probabilities that are the sum of two bf16 numbers, whatever the queries' type."""
    return ref.attend(q.float(), *args)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("shape", [(128, 1, 576, 512), (40, 1, 576, 512), (16, 1, 576, 512), (4, 2, 320, 64), (8, 2, 128, 128)])
@pytest.mark.parametrize("n", [1, 2, 3, 8, 40, 200])
def test_probabilities_of_two_parts(n, shape, dtype):
    """Values that cancel: what is left of them is far smaller than what one rounding of the probabilities to 8 bits moves.

    Queries of one channel each: a score is one product, so its own error leaves the bound tight.
    """
    Hq, Hkv, D, Dv = shape
    g = gen(21)
    kc, ks, kg, ksg = cache(n, Hkv, D, g)
    if Dv == 512:
        vc, vs, vg, vsg = kc[..., :Dv], ks[..., :Dv // 32], kg[..., :Dv], ksg[..., :Dv // 32]
    else:
        vc, vs, vg, vsg = cache(n, Hkv, Dv, g)
    q = torch.zeros(1, 1, Hq, D, dtype=dtype)
    q[0, 0, torch.arange(Hq), torch.randint(0, D, (Hq,), generator=g)] = (torch.randn(Hq, generator=g) * math.sqrt(D)).to(dtype)
    slots = torch.randperm(n, generator=g).to(torch.int32).view(1, 1, n)
    want = two_parts(q, kc, ks, vc, vs, [[slots[0, 0]]])
    out, lse = ets.attend_selected(q.to(dev()), kg, ksg, vg, vsg, slots.to(dev()))
    close(out, want[0], want[2], dtype)
    close(lse, want[1], want[3], FP32)


@pytest.mark.parametrize("n", [1500, 1900])  # 12 and 15 splits: the join's shares leave lanes over
@pytest.mark.parametrize("Dv", [32, 96, 128, 160, 192])
def test_joins_with_lanes_left_over(Dv, n):
    g = gen(22)
    kc, ks, kg, ksg = cache(n, 1, 64, g)
    vc, vs, vg, vsg = cache(n, 1, Dv, g)
    q = torch.randn(1, 1, 8, 64, generator=g).to(FP16)
    slots = torch.randperm(n, generator=g).to(torch.int32).view(1, 1, n)
    want = ref.attend(q, kc, ks, vc, vs, [[slots[0, 0]]])
    out, lse = ets.attend_selected(q.to(dev()), kg, ksg, vg, vsg, slots.to(dev()))
    close(out, want[0], want[2], FP16)
    close(lse, want[1], want[3], FP32)
