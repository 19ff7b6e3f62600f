"""The decode operators where a wave takes many steps: sizes that fill the device, sampled rows against tests/decode_reference.py.

With few lists each is dealt out until a wave has one step of it; these have as many lists, or keys, as make a wave go
on: through the steps, their slots' chunks, several heads of a workgroup, and from one sequence into the next.
"""
import pytest
import torch

import exact_top_selection_amd as ets
from tests import decode_reference as ref
from tests import dispatch_probe
from tests.test_gpu_step import BF16, FP16, FP32, cache, close, dev, gen, tree
from tests.test_gpu_step_edges import every_list, two_parts

pytestmark = pytest.mark.gpu


# sequences, query heads, cache heads, channels, slots of a list
LISTS = [
    (512, 8, 4, 128, 1100),   # four heads to a workgroup, 35 tiles a wave
    (512, 64, 4, 128, 300),   # the same with 16 rows a head
    (512, 6, 2, 64, 1100),    # two heads
    (512, 12, 6, 96, 1100),   # two of six
    (512, 2, 1, 128, 2200),   # one head, 18 tiles a wave, five chunks of slots
    (512, 20, 1, 64, 1500),   # two row tiles
    (512, 24, 1, 128, 700),
    (520, 4, 4, 192, 300),
    (300, 8, 4, 256, 700),    # one workgroup a compute unit
    (300, 80, 4, 256, 300),   # two row tiles of 256 channels, four heads
    (300, 20, 1, 256, 1100),
    (300, 20, 1, 224, 700),
    (300, 64, 1, 576, 1100),  # latent: values are the keys' first 512 channels
    (300, 20, 1, 576, 700),
    (150, 128, 1, 576, 500),
    (300, 4, 1, 320, 900),    # values apart from the keys
]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("case", LISTS)
def test_many_lists(case, far, dtype):
    """Lists with holes, each in its own order; far: sizes of keys over 2^12, so that references are raised along the way."""
    B, Hq, Hkv, D, n = case
    g = gen(31)
    S = n + 50
    x = torch.randn(S, Hkv, D, generator=g, dtype=torch.float64)
    if far:
        x = x * 2.0 ** (12 * torch.arange(S).double() / S - 4).view(S, 1, 1)
    kc, ks = ref.quantise(x)
    vc, vs = (kc[..., :512], ks[..., :16]) if D == 576 else ref.quantise(torch.randn(S, Hkv, D, generator=g).double())
    q = torch.randn(B, 1, Hq, D, generator=g).to(dtype)
    sample = [0, B // 3, B - 1]
    slots = torch.randint(-1, S, (B, 1, n), generator=g, dtype=torch.int32)
    slots[sample[0], 0] = torch.arange(n)              # all there, rising
    slots[sample[1], 0] = torch.arange(S - 1, S - 1 - n, -1)
    slots[sample[2], 0, n // 2:] = -1                  # the second half empty
    out, lse, want = every_list(q, kc, ks, vc, vs, slots, sample)
    close(out, want[0], want[2], dtype)
    close(lse, want[1], want[3], FP32)


SEQUENCES = [  # sequences, tokens, query heads, cache heads, channels, values' channels, positions, page
    (64, 9, 40, 8, 128, 128, 1100, 16),    # 45 rows a list in two groups, four heads
    (40, 5, 8, 2, 64, 64, 5000, 64),       # two heads, several chunks
    (300, 3, 5, 1, 96, 160, 1500, 48),
    (150, 4, 20, 1, 256, 256, 700, 100),   # 80 rows
    (300, 2, 40, 1, 576, 512, 700, 64),
    (300, 2, 8, 1, 320, 288, 500, 7),
]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("case", SEQUENCES)
def test_many_sequences_with_trees(case, dtype):
    B, T, Hq, Hkv, D, Dv, n, page = case
    g = gen(32)
    per = -(-(n + T) // page)
    pages = 2 * per
    kc, ks, kg, ksg = cache(pages * page, Hkv, D, g)
    vc, vs, vg, vsg = (kc[..., :Dv], ks[..., :Dv // 32], kg[..., :Dv], ksg[..., :Dv // 32]) if Dv == 512 else cache(pages * page, Hkv, Dv, g)
    table = torch.stack([torch.randperm(pages, generator=g)[:per] for _ in range(B)]).to(torch.int32)
    lens = torch.randint(n // 2, n + 1, (B,), generator=g).to(torch.int32)
    sample = [0, B // 2, B - 2, B - 1]
    lens[0], lens[B // 2], lens[B - 1] = n, 0, 1
    q = (torch.randn(B, T, Hq, D, generator=g)).to(dtype)
    drafts = torch.stack([ref.slots_of(table[b], page, int(lens[b]) + torch.arange(T)) for b in range(B)])
    mask = tree(B, T, g)
    out, lse = ets.attend_paged(q.to(dev()), kg, ksg, vg, vsg, table.to(dev()), lens.to(dev()), page, n,
                                tree_slots=drafts.to(torch.int32).to(dev()), tree_mask=mask.to(dev()))
    lists = [[ref.slots_of(table[b], page, torch.arange(int(lens[b])))] * T for b in sample]
    want = two_parts(q[sample], kc, ks, vc, vs, lists, drafts[sample], mask[sample])
    close(out[sample], want[0], want[2], dtype)
    close(lse[sample], want[1], want[3], FP32)


RUNS = [  # tokens, heads, channels, page, lengths
    (13, 64, 128, 64, [9000, 0, 0, 5000, 1, 30000, 0, 2049]),       # runs over several sequences, empty ones among them
    (1, 16, 64, 16, [(37 * i) % 301 for i in range(1000)]),         # several sequences to a counting lane
    (13, 64, 128, 64, [0, 150000, 130, 120001, 0]),                 # more than one piece of 2048 keys a workgroup
    (2, 128, 256, 48, [0, 70000, 33, 0, 60001]),
    (3, 5, 192, 7, [50000, 0, 100000]),
    (3, 17, 96, 100, [150001, 0, 0, 127]),
]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("case", RUNS)
def test_scores_of_long_runs(case, dtype):
    T, H, D, page, lens = case
    g = gen(33)
    B, L = len(lens), max(lens) + 3
    per = -(-L // page)
    pages = min(B * per, 3000)
    codes, scales, cg, sg = cache(pages * page, 1, D, g)
    table = torch.randint(0, pages, (B, per), generator=g, dtype=torch.int32)
    q, w = torch.randn(B, T, H, D, generator=g).to(dtype), torch.randn(B, T, H, generator=g)
    got = ets.index_scores(q.to(dev()), w.to(dev()), cg, sg, table.to(dev()), torch.tensor(lens, dtype=torch.int32, device=dev()), page, L)
    got = got.view(B, T, L)
    if B > 100:  # no score past a length is left out
        ends = torch.tensor(lens, device=dev()).view(B, 1, 1)
        assert torch.equal(got == -float("inf"), (torch.arange(L, device=dev()) >= ends).expand(B, T, L))
    rows = range(B) if B < 100 else [0, 1, 8, 500, 996, 999]
    for t in {0, T - 1}:
        for b in rows:
            want, bound = ref.index_scores(q[b:b + 1, t:t + 1], w[b:b + 1, t:t + 1], codes, scales, table[b:b + 1], lens[b:b + 1], page, L)
            close(got[b, t:t + 1], want, bound, FP32)


@pytest.mark.parametrize("layout,offset,R", [("half", 0, 128), ("interleaved", 64, 64), ("half", 3, 42)])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_large_outputs_equal_small_ones(layout, offset, R, dtype):
    """Outputs over 32 MiB are stored past the caches: the same bits as those of their parts."""
    g = gen(34)
    N, H, D = 5000, 40, 128
    x = torch.randn(N, H, D, generator=g).to(dtype).to(dev())
    pos = torch.randint(0, 1 << 20, (N,), generator=g, dtype=torch.int32).to(dev())
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=dev()) / R)
    whole = ets.rope(x, pos, freq, layout=layout, offset=offset)
    for at in range(0, N, 600):
        part = slice(at, min(at + 600, N))
        assert torch.equal(whole[part], ets.rope(x[part], pos[part], freq, layout=layout, offset=offset))
    codes, scales = torch.zeros(N, H, D, dtype=torch.uint8, device=dev()), torch.zeros(N, H, D // 32, dtype=torch.uint8, device=dev())
    slots = torch.randperm(N, generator=g).to(torch.int32).to(dev())
    ets.cache_write(x, slots, codes, scales)
    whole = ets.cache_read(codes, scales, slots, dtype=dtype)
    for at in range(0, N, 600):
        part = slice(at, min(at + 600, N))
        assert torch.equal(whole[part], ets.cache_read(codes, scales, slots[part], dtype=dtype))


def test_workgroups_go_round_the_xcds_from_wherever_the_last_launch_ended():
    """What the kernels' block numbering relies on in a process that has run grids of any size: block i shares an XCD with
    block i + X, though block 0 may stand on any."""
    cu, nx, _ = ets.device_limits()
    lib = dispatch_probe.load()
    x = torch.zeros(1, 1, 64, dtype=BF16, device=dev())
    pos, freq = torch.zeros(1, dtype=torch.int32, device=dev()), torch.ones(4, dtype=torch.float64, device=dev())
    for before in (0, 1, 3):
        for _ in range(before):
            ets.rope(x, pos, freq)  # one workgroup
        n = 2 * cu
        rec = torch.zeros((n, 4), dtype=torch.int64, device=dev())
        assert lib.ets_test_dispatch_probe(rec.data_ptr(), n, 500, 500, torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        xcc = rec[:, 0].cpu() & 0xF
        i = torch.arange(n)
        assert torch.equal(xcc, xcc[i % nx]) and xcc[:nx].sort().values.tolist() == list(range(nx))
