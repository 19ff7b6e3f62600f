"""The operators of a speculative step on the GPU against the plain 64-bit forms of tests/speculate_reference.py."""
import math
import random

import pytest
import torch

import exact_top_selection_amd as ets
from tests import decode_reference as ref
from tests import speculate_reference as spec
from tests.test_gpu_step import BF16, FP16, FP32, close, dev, gen
from tests.test_gpu_step_edges import close_where_numbers

pytestmark = pytest.mark.gpu


def ints(*values):
    return torch.tensor(values, dtype=torch.int32)


def filled(S, H, D, block, g, size=1.0):
    """A block cache of normal rows of differing size: (codes, scales) on the CPU, bytes."""
    x = torch.randn(S, H, D, generator=g, dtype=torch.float64) * torch.exp(torch.randn(S, H, 1, generator=g, dtype=torch.float64)) * size
    top = x.abs().view(S // block, block, H, D).amax((1, 3))
    m, p = torch.frexp(top)
    e = torch.where(m <= 0.875, p - 9, p - 8).clamp(spec.LOW, spec.HIGH)
    codes = spec.encode((x.view(S // block, block, H, D) * torch.exp2(-e.double())[:, None, :, None]).view(S, H, D))
    return codes, (e + 127).to(torch.uint8)


def pages(B, per, extra, g):
    """(page table of B sequences of `per` pages, pages of the cache), in random order."""
    return torch.randperm(B * per + extra, generator=g)[:B * per].to(torch.int32).view(B, per), B * per + extra


def same_codes(got, want):
    """Equal codes; the one that is no number has two of them."""
    got = got.view(torch.uint8).cpu()
    return bool(((got == want) | ((want & 127 == 127) & (got & 127 == 127))).all())


def tree(B, T, g):
    mask = torch.ones(B, T, dtype=torch.int64)
    for b in range(B):
        for t in range(1, T):
            parent = int(torch.randint(0, t, (1,), generator=g))
            bits = (int(mask[b, parent]) & ((1 << 64) - 1)) | 1 << t
            mask[b, t] = bits - (1 << 64) if bits >> 63 else bits
    return mask


# ---- block_write, block_keep

WRITE = [  # B, T, H, D, block, blocks of a page, pages of a sequence
    (1, 1, 1, 32, 1, 1, 2),
    (3, 1, 2, 128, 16, 1, 3),
    (2, 5, 3, 96, 4, 2, 3),
    (2, 70, 1, 64, 16, 3, 3),
    (2, 33, 2, 256, 100, 1, 2),     # a block beyond what lanes keep in registers
    (1, 130, 1, 256, 200, 1, 1),
    (4, 17, 2, 160, 8, 2, 2),
    (2, 9, 1, 128, 64, 1, 2),
]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("case", WRITE)
def test_block_write(case, dtype):
    B, T, H, D, block, per, M = case
    g = gen(41)
    page = block * per
    table, P = pages(B, M, 1, g)
    codes, scales = filled(P * page, H, D, block, g)
    for turn, size in enumerate((1.0, 30.0, 1e-3, 0.0, 5e4)):  # scales grow, and stay where values are small
        x = (torch.randn(B, T, H, D, generator=g) * size * torch.exp(torch.randn(B, T, H, 1, generator=g))).clamp(-6e4, 6e4).to(dtype)
        first = torch.randint(0, max(1, M * page - T + 2), (B,), generator=g, dtype=torch.int32)
        counts = torch.randint(0, T + 2, (B,), generator=g, dtype=torch.int32)
        if turn == 1:
            first[0], counts[0] = 0, T
        if turn == 2 and B > 1:
            first[1] = -1
        if turn == 4 and B > 2:
            table = table.clone()
            table[2, 0], table[1, -1] = -1, P
        want = spec.block_write(x, codes, scales, table, first, counts, page)
        got = codes.to(dev()).view(torch.float8_e4m3fn), scales.to(dev())
        ets.block_write(x.to(dev()), *got, table.to(dev()), first.to(dev()), counts.to(dev()), page)
        assert torch.equal(got[1].cpu(), want[1])
        assert torch.equal(got[0].view(torch.uint8).cpu(), want[0])
        codes, scales = want


def test_block_write_of_values_that_are_not_finite_and_borders():
    g = gen(42)
    codes, scales = filled(32, 2, 64, 8, g)
    x = torch.zeros(1, 24, 2, 64)
    x[0, 0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 3.0])
    x[0, 8, 0, 0] = math.nan                        # nothing finite but zeros
    x[0, 9, 1, 0] = math.inf
    x[0, 16, 0, :2] = torch.tensor([448 * 2.0 ** 5, -0.0])
    x[0, 17, 1, 0] = 448.5 * 2.0 ** 5               # just over the border
    table, at, n = ints(3, 0, 2, 1).view(1, 4), ints(0), ints(24)
    for dtype in (FP32, BF16):
        want = spec.block_write(x.to(dtype), codes, scales, table, at, n, 8)
        got = codes.to(dev()), scales.to(dev())
        ets.block_write(x.to(dtype).to(dev()), *got, table.to(dev()), at.to(dev()), n.to(dev()), 8)
        assert torch.equal(got[1].cpu(), want[1]) and want[1][0, 0] == 1 and want[1][2, 0] == 132
        assert same_codes(got[0], want[0])
    for size in (1e38, 3e38, 1e-40, 1e-45):  # exponents at the ends of their range
        y = torch.full((1, 3, 2, 64), size)
        want = spec.block_write(y, codes, scales, table, at, ints(3), 8)
        got = codes.to(dev()), scales.to(dev())
        ets.block_write(y.to(dev()), *got, table.to(dev()), at.to(dev()), ints(3).to(dev()), 8)
        assert torch.equal(got[1].cpu(), want[1]) and torch.equal(got[0].cpu(), want[0]), size


def test_block_write_strides_and_far_slots():
    g = gen(43)
    wide = torch.randn(3, 12, 5, 70, generator=g).to(BF16).to(dev())
    x = wide[:, ::2, 1:3, 3:67]
    big = torch.randint(0, 256, (48, 3, 101), generator=g, dtype=torch.uint8)
    codes, held = big[:, :2, 5:69], torch.randint(1, 247, (12, 7), generator=g, dtype=torch.uint8)
    table, first, counts = ints(5, 2, 0, 1, 3, 4).view(3, 2), ints(3, 0, 9), ints(6, 2, 6)
    want = spec.block_write(x.cpu(), codes, held[:, 1:5:3], table, first, counts, 8)
    there, scales = big.to(dev()), held.to(dev())
    ets.block_write(x, there[:, :2, 5:69], scales[:, 1:5:3], table.to(dev()), first.to(dev()), counts.to(dev()), 8)
    expect, bytes_ = big.clone(), held.clone()
    expect[:, :2, 5:69], bytes_[:, 1:5:3] = want
    assert torch.equal(scales.cpu(), bytes_) and same_codes(there[:, :2, 5:69], expect[:, :2, 5:69])
    there[:, :2, 5:69] = expect[:, :2, 5:69].to(dev())
    assert torch.equal(there.cpu(), expect)  # nothing beside the rows was written
    # slots whose place in memory passes 2^32 bytes
    far = torch.zeros((1 << 32) + (1 << 20), dtype=torch.uint8, device=dev())
    S = far.numel() // 2048
    codes, scales = far[:S * 2048].view(S, 8, 256), torch.full((S // 16, 8), 127, dtype=torch.uint8, device=dev())
    y = torch.randn(1, 20, 8, 256, generator=g)
    page = S // 16 - 2
    ets.block_write(y.to(dev()), codes, scales, ints(page, page + 1).view(1, 2).to(dev()), ints(3).to(dev()), ints(20).to(dev()), 16)
    small = torch.zeros(32, 8, 256, dtype=torch.uint8), torch.full((2, 8), 127, dtype=torch.uint8)
    want = spec.block_write(y, *small, ints(0, 1).view(1, 2), ints(3), ints(20), 16)
    assert torch.equal(codes[-32:].cpu(), want[0]) and torch.equal(scales[-2:].cpu(), want[1])
    assert int(far[:1 << 31].max()) == 0


KEEP = [  # B, T, H, D, block, blocks of a page, pages of a sequence
    (1, 1, 1, 32, 1, 1, 2),
    (4, 5, 2, 64, 4, 1, 4),
    (5, 24, 2, 128, 16, 2, 3),
    (3, 64, 1, 256, 8, 2, 6),
    (3, 40, 3, 96, 100, 1, 1),
    (6, 13, 8, 128, 1, 5, 6),
]


@pytest.mark.parametrize("case", KEEP)
def test_block_keep(case):
    B, T, H, D, block, per, M = case
    g, r = gen(44), random.Random(1)
    page = block * per
    table, P = pages(B, M, 0, g)
    codes, scales = filled(P * page, H, D, block, g)
    scales = (scales.int() + torch.randint(-6, 7, scales.shape, generator=g)).clamp(1, 246).to(torch.uint8)
    for turn in range(4):
        first = torch.randint(0, M * page - T + 1, (B,), generator=g, dtype=torch.int32)
        counts = torch.randint(0, T + 2, (B,), generator=g, dtype=torch.int32)
        path = torch.full((B, T), -1, dtype=torch.int32)
        for b in range(B):
            n = min(int(counts[b]), T)
            line = sorted(r.sample(range(T), n))
            if n and r.random() < 0.7:
                line[0] = 0
            path[b, :n] = torch.tensor(line, dtype=torch.int32)
        if turn == 1:
            path = path.flip(1).contiguous()  # any order, and entries that are no rows
        if turn == 2:
            path[0] = torch.arange(T)
            first[B - 1] = -3 if B > 1 else 0
        if turn == 3:
            path[0, 0], counts[0] = T - 1, 1
            table = table.clone()
            table[B - 1, M // 2] = P + 5
        want = spec.block_keep(codes, scales, table, first, path, counts, page)
        got = codes.to(dev()).view(torch.float8_e4m3fn), scales.to(dev())
        ets.block_keep(*got, table.to(dev()), first.to(dev()), path.to(dev()), counts.to(dev()), page)
        assert torch.equal(got[1].cpu(), want[1]), turn
        assert torch.equal(got[0].view(torch.uint8).cpu(), want[0]), turn
        codes, scales = want


def test_block_keep_keeps_every_code_and_scale():
    """Rows of all codes under scales at the ends of their range come back as they were, in a block of their own."""
    codes = torch.zeros(48, 1, 256, dtype=torch.uint8)
    codes[40] = torch.arange(256, dtype=torch.uint8)
    for byte in (1, 2, 119, 245, 246):
        scales = torch.full((6, 1), byte, dtype=torch.uint8)
        got = codes.to(dev()), scales.to(dev())
        ets.block_keep(*got, torch.arange(6, dtype=torch.int32).view(1, 6).to(dev()), ints(8).to(dev()),
                       ints(*([32] + [0] * 39)).view(1, 40).to(dev()), ints(1).to(dev()), 8)
        assert int(got[1][1, 0]) == byte
        back, want = got[0].cpu()[8, 0], codes[40, 0]
        none = want & 127 == 127
        assert torch.equal(back[~none], want[~none]) and (back[none] & 127 == 127).all()


# ---- attend_blocks

ATTEND = [  # B, T, Hq, Hkv, D, Dv, L, block, blocks of a page, form
    (1, 1, 1, 1, 32, 32, 1, 1, 1, "all"),
    (2, 1, 8, 2, 128, 128, 100, 16, 1, "all"),
    (1, 3, 6, 2, 64, 64, 65, 8, 2, "all"),
    (2, 1, 4, 4, 96, 160, 77, 4, 3, "all"),
    (1, 2, 40, 1, 192, 192, 40, 64, 1, "all"),
    (2, 1, 32, 8, 256, 256, 200, 100, 1, "all"),
    (1, 1, 16, 1, 128, 128, 2000, 64, 1, "all"),   # many splits
    (3, 5, 8, 2, 128, 128, 70, 16, 1, "causal"),
    (2, 40, 4, 1, 64, 64, 90, 16, 2, "causal"),
    (1, 200, 4, 2, 128, 128, 333, 32, 2, "causal"),
    (2, 33, 3, 1, 96, 64, 33, 8, 1, "causal"),     # nothing before the tokens
    (1, 100, 2, 2, 256, 256, 150, 64, 1, "causal"),
    (2, 13, 8, 4, 96, 96, 120, 16, 3, "tree"),
    (2, 64, 2, 1, 128, 128, 130, 16, 1, "tree"),
    (1, 7, 20, 1, 192, 128, 40, 1, 1, "tree"),
    (3, 2, 4, 4, 64, 256, 50, 100, 1, "tree"),
]


def block_case(case, dtype, seed=45):
    B, T, Hq, Hkv, D, Dv, L, block, per, form = case
    g = gen(seed)
    page = block * per
    table, P = pages(B, -(-L // page), 2, g)
    kc, ks = filled(P * page, Hkv, D, block, g)
    vc, vs = filled(P * page, Hkv, Dv, block, g)
    q = torch.randn(B, T, Hq, D, generator=g).to(dtype)
    lens = torch.randint(max(1, min(T, L) if form != "all" else 1), L + 1, (B,), generator=g, dtype=torch.int32)
    lens[0] = L
    first = mask = None
    if form != "all":
        first = (lens - T).clamp(min=0)
        if B > 1:
            first[1] += T // 2  # its last tokens are padding
    if form == "tree":
        mask = tree(B, T, g)
    return q, kc, ks, vc, vs, table, lens, page, L, first, mask


def run_blocks(q, kc, ks, vc, vs, table, lens, page, L, first, mask, **kw):
    on = lambda t: None if t is None else t.to(dev())  # noqa: E731
    return ets.attend_blocks(on(q), on(kc), on(ks), on(vc), on(vs), on(table), on(lens), page, L, first=on(first), tree_mask=on(mask), **kw)


def check_blocks(case, dtype):
    q, kc, ks, vc, vs, table, lens, page, L, first, mask = case
    lists = spec.seen(table, page, kc.shape[0] // page, lens, L, q.shape[1], first, mask)
    want = spec.attend(q, kc, ks, vc, vs, lists)
    out, lse = run_blocks(*case)
    value, bound = want[0], want[2]
    if dtype == FP16:
        # results from 65520 on (the largest number, 65504, and half its step) are infinite in fp16; those within their
        # bound of that may be either
        border = (value.abs() - 65520).abs() <= bound
        out = out.masked_fill(border.to(dev()), 0)
        value = torch.where(border, 0.0, torch.where(value.abs() > 65520, value.sign() * math.inf, value))
        bound = torch.where(border | torch.isinf(value), 0.0, bound)
    close_where_numbers(out, value, bound, dtype)
    close_where_numbers(lse, want[1], want[3], FP32)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("case", ATTEND)
def test_attend_blocks(case, dtype):
    check_blocks(block_case(case, dtype), dtype)


@pytest.mark.parametrize("form", ["all", "causal", "tree"])
def test_attend_blocks_bad_pages_and_lengths(form):
    case = list(block_case((4, 6, 4, 2, 64, 64, 90, 8, 2, form), BF16))
    q, kc, ks, vc, vs, table, lens, page, L, first, mask = case
    P = kc.shape[0] // page
    table[0, 1], table[1, 0], table[2, 3], table[2, 0] = -1, P, 0x7FFFFFFF, -0x7FFFFFFF
    lens[1], lens[3] = 0x7FFFFFFF, 0
    if first is not None:
        first[2] = -2
        first[1] = 84
    check_blocks(case, BF16)
    lens[:] = -5
    out, lse = run_blocks(*case)
    assert not out.any() and torch.isinf(lse).all()


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("shape", [(8, 2, 64, 64, 5), (12, 2, 128, 96, 40), (4, 1, 192, 192, 5), (3, 1, 256, 256, 64), (4, 4, 128, 128, 1)])
@pytest.mark.parametrize("form", ["causal", "tree"])
def test_rows_that_are_no_numbers(form, shape, dtype):
    """What a token does not see does not reach it: rows of drafts beside its line, of later tokens, behind the length."""
    Hq, Hkv, D, Dv, T = shape
    case = block_case((2, T, Hq, Hkv, D, Dv, 70 + T, 8, 2, form), dtype, seed=46)
    q, kc, ks, vc, vs, table, lens, page, L, first, mask = case
    lens[:] = ints(60 + T, 70 + T)
    first[:] = lens - T
    P = kc.shape[0] // page
    at = lambda b, p: spec.place(table[b], page, P, p)  # noqa: E731
    vc[at(0, 60 + T // 2), 0, 5], vc[at(1, 70 + T - 1), -1, Dv - 1] = 0x7F, 0xFF
    if T > 2:
        kc[at(1, 70 + T - 2), 0, 0] = 0x7F
    for p in range(60 + T, -(-(60 + T) // 8) * 8):  # never written
        kc[at(0, p)], vc[at(0, p)] = 0xFF, 0x7F
    lists = spec.seen(table, page, P, lens, L, T, first, mask)
    want = spec.attend(q, kc, ks, vc, vs, lists)
    assert T == 1 or torch.isfinite(want[0][:, 0]).all()
    check_blocks(case, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("T,Hq,D", [(1, 16, 128), (1, 2, 64), (40, 4, 256), (70, 2, 64)])
def test_attend_blocks_of_scores_far_apart(T, Hq, D, order, dtype):
    """Scores pass each other by far more than the softmax's reference lags, in either direction; values of all sizes."""
    g, n, block = gen(47), 400, 16
    x = torch.zeros(n, 1, D, dtype=torch.float64)
    at = {"rising": torch.arange(n), "falling": torch.arange(n).flip(0), "mixed": torch.randperm(n, generator=g)}[order]
    x[:, 0, 0] = at.double() / n * 400 - 200
    codes = torch.zeros(n, 1, D, dtype=torch.uint8)
    scales = torch.full((n // block, 1), 127, dtype=torch.uint8)
    codes[:, :, 0] = spec.encode(x[:, :, 0])
    vc, vs = filled(n, 1, D, block, g)
    vs = (vs.int() + torch.randint(-40, 41, vs.shape, generator=g)).clamp(1, 246).to(torch.uint8)
    q = torch.zeros(1, T, Hq, D)
    q[..., 0] = torch.randn(1, T, Hq, generator=g) * math.sqrt(D) / 2
    table, lens = torch.arange(n // block, dtype=torch.int32).view(1, -1), ints(n)
    first = ints(n - T) if T > 1 else None
    check_blocks((q.to(dtype), codes, scales, vc, vs, table, lens, block, n, first, None), dtype)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("shape", [(16, 2, 128, 128, 1), (4, 1, 64, 64, 40), (8, 8, 256, 192, 1)])
@pytest.mark.parametrize("n", [1, 2, 3, 8, 40, 200])
def test_probabilities_of_two_parts(n, shape, dtype):
    """Values that cancel: what is left of them is far smaller than what a rounding of the probabilities to 8 bits moves."""
    Hq, Hkv, D, Dv, T = shape
    g = gen(48)
    kc, ks = filled(256, Hkv, D, 8, g)
    vc, vs = filled(256, Hkv, Dv, 8, g)
    q = torch.zeros(1, T, Hq, D, dtype=dtype)
    q[0, :, torch.arange(Hq), torch.randint(0, D, (Hq,), generator=g)] = (torch.randn(T, Hq, generator=g) * math.sqrt(D)).to(dtype)
    table = torch.randperm(16, generator=g).to(torch.int32).view(1, 16)
    check_blocks((q, kc, ks, vc, vs, table, ints(n), 16, 256, ints(max(0, n - T)) if T > 1 else None, None), dtype)


def test_attend_blocks_strides_streams_and_workspace():
    case = block_case((2, 3, 8, 2, 128, 64, 150, 8, 2, "causal"), BF16)
    q, kc, ks, vc, vs, table, lens, page, L, first, _ = case
    plain = run_blocks(*case)
    S = kc.shape[0]
    wq = torch.zeros(2, 5, 9, 141, dtype=BF16, device=dev())
    wq[:, 1:4, :8, 3:131] = q.to(dev())
    both = torch.full((S, 3, 203), 255, dtype=torch.uint8, device=dev())
    both[:, :2, 1:129], both[:, :2, 130:194] = kc.to(dev()), vc.to(dev())
    bytes_ = torch.zeros(S // 8, 5, dtype=torch.uint8, device=dev())
    bytes_[:, 0:3:2], bytes_[:, 1:4:2] = ks.to(dev()), vs.to(dev())
    wide = torch.full((2, table.shape[1] + 3), -1, dtype=torch.int32, device=dev())
    wide[:, :table.shape[1]] = table.to(dev())
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        space = torch.full((1 << 24,), 255, dtype=torch.uint8, device=dev())
        got = ets.attend_blocks(wq[:, 1:4, :8, 3:131], both[:, :2, 1:129], bytes_[:, 0:3:2], both[:, :2, 130:194], bytes_[:, 1:4:2],
                                wide, lens.to(dev()), page, L, first=first.to(dev()), workspace=space)
    torch.cuda.synchronize()
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
    with pytest.raises(ValueError, match="workspace"):
        run_blocks(*case, workspace=space[:16])


def test_attend_blocks_far_slots():
    """Slots whose place in memory passes 2^32 bytes."""
    g = gen(49)
    far = torch.zeros((1 << 32) + (1 << 20), dtype=torch.uint8, device=dev())
    S = far.numel() // 2048
    codes, scales = far[:S * 2048].view(S, 8, 256), torch.full((S // 16, 8), 127, dtype=torch.uint8, device=dev())
    kc, ks = filled(64, 8, 256, 16, g)
    codes[-64:], scales[-4:] = kc.to(dev()), ks.to(dev())
    q = torch.randn(1, 2, 16, 256, generator=g).to(BF16)
    table = torch.arange(4, dtype=torch.int32).view(1, 4)
    got = ets.attend_blocks(q.to(dev()), codes, scales, codes, scales, (table + (S // 16 - 4)).to(dev()), ints(60).to(dev()), 16, 64)
    want = run_blocks(q, kc, ks, kc, ks, table, ints(60), 16, 64, None, None)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("size", [112, 0, -90])  # powers of two: values to 448 * 2^112, and to 2^-90
@pytest.mark.parametrize("order", ["rising", "falling"])
@pytest.mark.parametrize("Hq,D", [(4, 64), (2, 128), (3, 192), (2, 256)])
def test_values_near_the_ends_of_the_range(Hq, D, order, size, T):
    """Scores pass each other by up to 2^20 while values stand near either end of what sums can hold."""
    g, n = gen(60), 400
    kc, ks = torch.zeros(n, 1, D, dtype=torch.uint8), torch.full((n // 8, 1), 127, dtype=torch.uint8)
    at = torch.arange(n) if order == "rising" else torch.arange(n).flip(0)
    kc[:, 0, 0] = spec.encode(at.double() / n * 40 - 20)
    vc, vs = filled(n, 1, D, 8, g)
    vc = vc & 0x7F if size == 112 else vc  # nothing cancels
    vs = (vs.int() - vs.int().max() + 127 + size - (8 if size < 0 else 0)).clamp(1, 246).to(torch.uint8)
    q = torch.zeros(1, T, Hq, D)
    q[..., 0] = (torch.arange(T * Hq).view(1, T, Hq) % 5 - 2) / 2 * math.sqrt(D) / math.log2(math.e)
    table = torch.arange(n // 8, dtype=torch.int32).view(1, -1)
    check_blocks((q.to(BF16), kc, ks, vc, vs, table, ints(n), 8, n, ints(n - T) if T > 1 else None, None), BF16)


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("behind", [True, False])
def test_scores_of_minus_infinity(behind, T):
    """Keys whose score leaves the 32-bit range: alone they are nothing, before others they weigh nothing."""
    g, n, D = gen(61), 200, 64
    kc, ks = torch.zeros(n, 1, D, dtype=torch.uint8), torch.full((n // 8, 1), 246, dtype=torch.uint8)
    kc[:, 0, 0] = 0x7E
    if behind:
        ks[160 // 8:] = 1
    vc, vs = filled(n, 1, D, 8, g)
    q = torch.zeros(1, T, 2, D)
    q[..., 0] = -3e4
    table = torch.arange(n // 8, dtype=torch.int32).view(1, -1)
    out, lse = run_blocks(q.to(BF16), kc, ks, vc, vs, table, ints(n), 8, n, ints(n - T) if T > 1 else None, None)
    if not behind:
        assert not out.any() and (lse == -math.inf).all()
        return
    sees = [torch.arange(160, n if T == 1 else n - T + t + 1) for t in range(T)]
    want = spec.attend(q.to(BF16), kc, ks, vc, vs, [sees])
    close(out, want[0], want[2], BF16)
    close(lse, want[1], want[3], FP32)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("B,T,Hq,Hkv,D,L", [(32, 256, 16, 16, 64, 300), (32, 130, 32, 16, 128, 200),  # for several turns of the device
                                            (1, 100, 8, 8, 64, 64), (1, 64, 3, 3, 128, 200), (9, 33, 1, 1, 256, 900),
                                            (5, 70, 6, 3, 192, 150), (70, 1, 8, 8, 128, 700)])
def test_attend_blocks_of_many_lists(B, T, Hq, Hkv, D, L, dtype):
    """Batches that fill the device in its different ways; some rows of them next to the formula."""
    g = gen(62)
    table, P = pages(B, -(-L // 16), 1, g)
    kc, ks = filled(P * 16, Hkv, D, 16, g)
    vc, vs = filled(P * 16, Hkv, D, 16, g)
    q = torch.randn(B, T, Hq, D, generator=g).to(dtype)
    lens = torch.randint(max(1, L // 2), L + 1, (B,), generator=g, dtype=torch.int32)
    first = lens - T // 2  # half of the tokens are padding
    out, lse = run_blocks(q, kc, ks, vc, vs, table, lens, 16, L, first if T > 1 else None, None)
    G = Hq // Hkv
    for b in {0, B // 2, B - 1}:
        for h in {0, Hkv - 1}:
            lists = spec.seen(table[b:b + 1], 16, P, lens[b:b + 1], L, T, first[b:b + 1] if T > 1 else None)
            some = sorted({0, 1, T // 3, T // 2 - 1, T // 2, T - 1} & set(range(T)))
            want = spec.attend(q[b:b + 1, some, h * G:h * G + G], kc[:, h:h + 1], ks[:, h:h + 1], vc[:, h:h + 1], vs[:, h:h + 1],
                               [[lists[0][t] for t in some]])
            close(out[b:b + 1, some, h * G:h * G + G], want[0], want[2], dtype)
            close(lse[b:b + 1, some, h * G:h * G + G], want[1], want[3], FP32)
    assert torch.equal(out, run_blocks(q, kc, ks, vc, vs, table, lens, 16, L, first if T > 1 else None, None)[0])


# ---- verify_drafts

def check_verify(probs, tokens, uniform, draft=None, mask=None, lens=None):
    want = spec.verify(probs, tokens, uniform, draft, mask, lens)
    on = lambda t: None if t is None else t.to(dev())  # noqa: E731
    got = ets.verify_drafts(on(probs), on(tokens), on(uniform), draft_probs=on(draft), tree_mask=on(mask), lens=on(lens))
    for name, a, b in zip(("tokens", "path", "counts"), got, want):
        assert torch.equal(a.cpu(), b), name
    return want


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("form", ["draft", "chain", "tree"])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (40, 6, 50), (6, 64, 20), (3, 5, 4096), (2, 4, 4097), (3, 9, 20011), (2, 3, 9000)])
def test_verify(B, T, V, form, dtype):
    g = gen(50)
    for turn in range(3):
        probs = torch.softmax(3 * torch.randn(B, T, V, generator=g), -1).to(dtype)
        draft = None
        if form == "draft":
            near = probs[:, :T - 1].float() * torch.exp(0.5 * torch.randn(B, T - 1, V, generator=g))
            draft = (near / near.sum(-1, keepdim=True)).to(dtype)
        mask = tree(B, T, g) if form == "tree" else None
        tokens = torch.randint(0, V, (B, T), generator=g, dtype=torch.int32)
        above = torch.tensor([[t - 1 if mask is None else max(0, (int(mask[b, t]) & ((1 << t) - 1)).bit_length() - 1) for t in range(T)]
                              for b in range(B)])
        for t in range(1, T):
            for b in range(B):
                row = (draft[b, t - 1] if draft is not None else probs[b, above[b, t]]).float()
                tokens[b, t] = int(torch.multinomial(row, 1, generator=g))
        uniform = torch.rand(B, T, generator=g) * (0.4 if form != "draft" else 1.0)
        if turn == 1:
            uniform[0, 0], tokens[0, T // 2] = 0.0, -1
            uniform[B - 1, T - 1] = 1 - 2.0 ** -24
            tokens[B - 1, T - 1] = V
        lens = None if turn == 0 else torch.randint(-1 if turn == 2 else 1, T + 2, (B,), generator=g, dtype=torch.int32)
        want = check_verify(probs, tokens, uniform, draft, mask, lens)
        if B == 40:
            assert int(want[2].max()) > 2 and int(want[2].min()) <= 1


def test_verify_takes_all_or_nothing():
    """One-hot rows (a greedy target), equal draft and target, rows of zeros, and random numbers outside [0, 1)."""
    T, V = 5, 70
    probs = torch.zeros(4, T, V)
    tokens = torch.arange(4 * T, dtype=torch.int32).view(4, T) % V
    for t in range(T - 1):
        probs[0, t, tokens[0, t + 1]] = 1      # all taken
        probs[1, t, tokens[1, t + 1] + 30] = 1  # none taken
    probs[0, T - 1, 69], probs[1, T - 1, 0] = 1, 1
    probs[2] = 1.0 / 64                        # equal weights: the mark falls on whole numbers of them
    uniform = torch.full((4, T), 0.5)
    want = check_verify(probs, tokens, uniform)
    assert want[2].tolist() == [T, 1, 1, 1] and want[0][0].tolist() == [1, 2, 3, 4, 69] and int(want[0][3, 0]) == -1
    same = torch.softmax(torch.randn(4, T, V, generator=gen(51)), -1)
    want = check_verify(same, tokens, torch.full((4, T), 1 - 2.0 ** -24), draft=same[:, :-1].contiguous())
    assert (want[2] == T).all()  # u < 1
    want = check_verify(same, tokens, torch.full((4, T), 1.0), draft=same[:, :-1].contiguous())
    assert (want[2] == 1).all()  # refused, and nothing of max(p - q, 0) is left: drawn from p itself
    for u in (0.0, -1.0, 1.0, 2.0, math.nan, math.inf):
        odd = same.clone()
        odd[0, :, 3], odd[1, :, 5], odd[2, :, 60:], odd[3, 0, :] = math.nan, math.inf, 0.0, -1.0
        check_verify(odd, tokens, torch.full((4, T), u))
        check_verify(odd, tokens, torch.full((4, T), u), draft=same[:, :-1].contiguous())


def test_verify_twins_and_lost_nodes():
    """Siblings of the same token, nodes that hang on nothing, bits of later nodes and of the node itself."""
    g = gen(52)
    T, V = 8, 30
    probs = torch.softmax(torch.randn(16, T, V, generator=g), -1)
    tokens = torch.randint(0, 4, (16, T), generator=g, dtype=torch.int32)
    mask = torch.tensor([1, 1, 1 | 2, 5, 0, 1 | 1 << 4, -1, 1 << 7]).repeat(16, 1)
    for _ in range(4):
        check_verify(probs, tokens, torch.rand(16, T, generator=g) * 0.3, mask=mask)


def test_verify_strides_and_streams():
    g = gen(53)
    B, T, V = 3, 4, 5001
    probs = torch.softmax(torch.randn(B, T, V, generator=g), -1).to(BF16)
    draft = torch.softmax(torch.randn(B, T - 1, V, generator=g), -1).to(BF16)
    tokens, uniform = torch.randint(0, V, (B, T), generator=g, dtype=torch.int32), torch.rand(B, T, generator=g)
    want = spec.verify(probs, tokens, uniform, draft)
    wide = torch.full((B, T + 2, V + 7), math.nan, dtype=BF16, device=dev())
    wide[:, 1:T + 1, 3:V + 3] = probs.to(dev())
    both = torch.full((T - 1, B, V + 1), math.nan, dtype=BF16, device=dev())
    both[..., 1:] = draft.transpose(0, 1).to(dev())
    wt, wu = torch.zeros(B, 2 * T, dtype=torch.int32, device=dev()), torch.zeros(B, T + 1, device=dev())
    wt[:, :T], wu[:, :T] = tokens.to(dev()), uniform.to(dev())
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        space = torch.full((1 << 16,), 255, dtype=torch.uint8, device=dev())
        got = ets.verify_drafts(wide[:, 1:T + 1, 3:V + 3], wt[:, :T], wu[:, :T], draft_probs=both.transpose(0, 1)[..., 1:],
                                workspace=space)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.cpu(), b)


# ---- pages

def pool(P, B, M, share, g):
    """(refs, table) of a pool in use by rows of differing length, some pages held by several."""
    table = torch.full((B, M), -1, dtype=torch.int32)
    order = torch.randperm(P, generator=g).tolist()
    refs = torch.zeros(P, dtype=torch.int32)
    for b in range(B):
        for j in range(int(torch.randint(0, M + 1, (1,), generator=g))):
            if torch.rand(1, generator=g) < 0.2 and b:
                e = int(table[b - 1, j])
            else:
                e = order.pop() if len(order) > P * (1 - share) else -1
            if e < 0:
                break
            table[b, j] = e
            refs[e] += 1
    return refs, table


POOLS = [(1, 1, 1, 4), (7, 3, 4, 1), (100, 8, 10, 16), (5000, 40, 60, 64), (20000, 100, 90, 3), (4096, 5, 1000, 8)]  # P, B, M, page


@pytest.mark.parametrize("P,B,M,page", POOLS)
def test_pages_extend_and_free(P, B, M, page):
    g = gen(54)
    refs, table = pool(P, B, M, 0.7, g)
    if B > 2:
        table[1, M // 2], table[2, M - 1] = -7, P  # no pages either
    got, rows = refs.to(dev()), table.to(dev())
    for turn in range(4):
        refs, table = got.cpu(), rows.cpu()
        lens = torch.randint(-3, M * page + 2 * page, (B,), generator=g, dtype=torch.int32)
        want = spec.extend(refs, table, lens, page)
        lacking = ets.pages_extend(got, rows, lens.to(dev()), page)
        assert got.tolist() == want[0] and rows.tolist() == want[1] and lacking.tolist() == want[2]
        lens = torch.randint(-3, M * page + 2, (B,), generator=g, dtype=torch.int32)
        refs, table = got.cpu(), rows.cpu()
        want = spec.release(refs, table, lens, page)
        ets.pages_free(got, rows, lens.to(dev()), page)
        assert got.tolist() == want[0] and rows.tolist() == want[1]


def held(P, page, g):
    """Buffers of several page sizes, odd ones among them."""
    return [torch.randint(0, 256, shape, generator=g, dtype=torch.uint8)
            for shape in ((P * page, 2, 33), (P, 3), (P * 2, 16), (P, 70000 // P + 5))] + [torch.randn(P * page, 5, generator=g)]


def same_pages(got, buffers, pairs, P):
    for a, b in zip(got, buffers):
        want = b.clone().view(P, -1)
        old = b.view(P, -1)
        for s, d in pairs:
            want[d] = old[s]
        assert torch.equal(a.cpu().view(P, -1), want)


@pytest.mark.parametrize("P,B,M,page", POOLS)
def test_pages_fork(P, B, M, page):
    g = gen(55)
    for share in (0.5, 0.97):
        refs, table = pool(P, B, M, share, g)
        if B > 2:
            table[2, 0] = P + 1
        n = 2 * B + 1
        lens = torch.randint(-2, M * page + page, (B,), generator=g, dtype=torch.int32)
        parents = torch.randint(-1, B + 1, (n,), generator=g, dtype=torch.int32)
        buffers = held(P, page, g)
        on = [t.to(dev()) for t in buffers]
        for wide in (M, M + 2, max(1, M - 1)):
            want = spec.fork(refs, table, lens, page, parents, wide)
            got, rows = refs.to(dev()), torch.full((n, wide + 3), 99, dtype=torch.int32, device=dev())
            out, lacking = ets.pages_fork(got, table.to(dev()), lens.to(dev()), page, parents.to(dev()), on, out=rows[:, :wide])
            assert got.tolist() == want[0] and out.tolist() == want[1] and lacking.tolist() == want[2]
            assert (rows[:, wide:] == 99).all()
            same_pages(on, buffers, want[3], P)
            buffers = [t.cpu() for t in on]


@pytest.mark.parametrize("P,B,M,page", POOLS)
def test_pages_compact(P, B, M, page):
    g = gen(56)
    for share in (0.0, 0.4, 0.9, 1.0):
        refs, table = pool(P, B, M, share, g)
        if share == 1.0:
            refs = refs.clamp(min=1)
        elif B > 2 and P > 50:
            table[1, 0], table[2, 1] = P, int((refs <= 0).nonzero()[-1])  # no page, a free page
        buffers = held(P, page, g)
        want = spec.compact(refs, table)
        got, rows, on = refs.to(dev()), table.to(dev()), [t.to(dev()) for t in buffers]
        moved = ets.pages_compact(got, rows, on)
        assert got.tolist() == want[0] and rows.tolist() == want[1] and moved.tolist() == want[2]
        same_pages(on, buffers, want[3], P)


def test_pages_copy():
    g = gen(57)
    P = 50
    buffers = held(P, 4, g)
    on = [t.to(dev()) for t in buffers]
    order = torch.randperm(P, generator=g).to(torch.int32)
    src, dst = order[:20].clone(), order[20:40].clone()
    src[3], dst[4], src[5], dst[6] = -1, P, P, -9
    ets.pages_copy(on, src.to(dev()), dst.to(dev()), P)
    same_pages(on, buffers, [(s, d) for s, d in zip(src.tolist(), dst.tolist()) if 0 <= s < P and 0 <= d < P], P)
    ets.pages_copy([], src.to(dev()), dst.to(dev()), P)
    ets.pages_copy(on, src[:0].to(dev()), dst[:0].to(dev()), P)
    # a page whose place passes 2^32 bytes
    far = torch.zeros(3, (1 << 31) + 5, dtype=torch.uint8, device=dev())
    far[0, -100:] = torch.arange(100, dtype=torch.uint8, device=dev())
    ets.pages_copy([far], ints(0).to(dev()), ints(2).to(dev()), 3)
    assert torch.equal(far[2, -100:], far[0, -100:]) and int(far[1].max()) == 0 and int(far[2, :-100].max()) == 0


def test_empty_calls():
    new = dict(device=dev())
    refs, table, none = torch.zeros(0, dtype=torch.int32, **new), torch.full((2, 3), -1, dtype=torch.int32, **new), torch.zeros(0, dtype=torch.int32, **new)
    assert ets.pages_extend(refs, table, ints(9, 1).to(dev()), 4).tolist() == [3, 1]
    ets.pages_free(refs, table, ints(0, 0).to(dev()), 4)
    rows, lacking = ets.pages_fork(refs, table, ints(9, 1).to(dev()), 4, ints(0, 1).to(dev()))
    assert (rows == -1).all() and lacking.tolist() == [0, 0]
    assert ets.pages_compact(refs, table).numel() == 0
    full = torch.ones(4, dtype=torch.int32, **new)
    assert ets.pages_extend(full, table[:0], none, 4).numel() == 0
    assert ets.pages_fork(full, table[:0], none, 4, none)[0].shape == (0, 3)
    assert ets.pages_compact(full, table[:, :0]).tolist() == [0, 1, 2, 3]
    codes, scales = torch.zeros(0, 2, 64, dtype=torch.uint8, **new), torch.zeros(0, 2, dtype=torch.uint8, **new)
    x = torch.zeros(2, 3, 2, 64, dtype=BF16, **new)
    ets.block_write(x, codes, scales, table, ints(0, 0).to(dev()), ints(3, 3).to(dev()), 4)
    ets.block_keep(codes, scales, table, ints(0, 0).to(dev()), torch.full((2, 3), 2, dtype=torch.int32, **new), ints(3, 3).to(dev()), 4)
    out, lse = ets.attend_blocks(x, codes, scales, codes, scales, table, ints(5, 0).to(dev()), 4, 12)
    assert not out.any() and torch.isinf(lse).all()
    out, lse = ets.attend_blocks(x[:, :0], codes, scales, codes, scales, table, ints(5, 0).to(dev()), 4, 12)
    assert out.shape == (2, 0, 2, 64)
    assert ets.verify_drafts(torch.zeros(0, 2, 5, **new), table[:0, :2], torch.zeros(0, 2, **new))[0].shape == (0, 2)


# ---- together

def test_a_step_in_a_graph():
    """A speculative step captured once: pages taken, drafts written, attended, verified, kept, pages let go.  Each replay,
    with new inputs and eager work between, leaves what the eager step leaves."""
    g = gen(58)
    B, T, H, D, V, page, block, M = 4, 6, 2, 64, 300, 8, 4, 20
    P = B * M
    mask = tree(B, T, g).to(dev())

    def state():
        return dict(codes=torch.zeros(P * page, H, D, dtype=torch.uint8, device=dev()), scales=torch.full((P * page // block, H), 127, dtype=torch.uint8, device=dev()),
                    refs=torch.zeros(P, dtype=torch.int32, device=dev()), table=torch.full((B, M), -1, dtype=torch.int32, device=dev()),
                    lens=torch.zeros(B, dtype=torch.int32, device=dev()), root=torch.zeros(B, dtype=torch.int32, device=dev()))

    x = torch.zeros(B, T, H, D, dtype=BF16, device=dev())
    q = torch.zeros(B, T, 4 * H, D, dtype=BF16, device=dev())
    probs = torch.zeros(B, T, V, device=dev())
    tokens = torch.zeros(B, T, dtype=torch.int32, device=dev())
    uniform = torch.zeros(B, T, device=dev())
    all_rows = torch.full((B,), T, dtype=torch.int32, device=dev())

    def step(s):
        reach = s["lens"] + T
        lacking = ets.pages_extend(s["refs"], s["table"], reach, page)
        ets.block_write(x, s["codes"], s["scales"], s["table"], s["lens"], all_rows, page)
        out, lse = ets.attend_blocks(q, s["codes"], s["scales"], s["codes"], s["scales"], s["table"], reach, page, M * page, first=s["lens"],
                                     tree_mask=mask)
        tokens[:, 0] = s["root"]
        new, path, counts = ets.verify_drafts(probs, tokens, uniform, tree_mask=mask)
        ets.block_keep(s["codes"], s["scales"], s["table"], s["lens"], path, counts, page)
        s["lens"] += counts
        s["root"].copy_(new.gather(1, (counts - 1).long().view(-1, 1))[:, 0])
        ets.pages_free(s["refs"], s["table"], s["lens"], page)
        branch, short = ets.pages_fork(s["refs"], s["table"], s["lens"], page, all_rows - T, [s["codes"], s["scales"]])
        ets.pages_free(s["refs"], branch, all_rows - T, page)
        moved = ets.pages_compact(s["refs"], s["table"], [s["codes"], s["scales"]])
        return lacking, out, lse, new, path, counts, short, moved

    step(state())  # warm
    a, b = state(), state()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            kept = step(a)
    longest = 0
    for rep in range(8):
        x.copy_(torch.randn(B, T, H, D, generator=g).to(BF16))
        q.copy_(torch.randn(B, T, 4 * H, D, generator=g).to(BF16))
        probs.copy_(torch.softmax(3 * torch.randn(B, T, V, generator=g), -1))
        tokens.copy_(probs.cpu()[:, :1].expand(B, T, V).reshape(-1, V).multinomial(1, generator=g).view(B, T).to(torch.int32))
        uniform.copy_(torch.rand(B, T, generator=g) * 0.2)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in kept]
        want = step(b)
        for i, (c, d) in enumerate(zip(got, want)):
            assert torch.equal(c, d), (rep, i)
        for name in a:
            assert torch.equal(a[name], b[name]), (rep, name)
        assert int(got[0].sum()) == 0 and int((a["refs"] > 0).sum()) == int(((a["lens"] + page - 1) // page).sum())
        longest = max(longest, int(got[5].max()))
        torch.cuda.synchronize()
    assert longest > 1


def test_refusals():
    g = gen(59)
    new = dict(device=dev())
    codes, scales = torch.zeros(16, 2, 64, dtype=torch.uint8, **new), torch.full((4, 2), 127, dtype=torch.uint8, **new)
    x = torch.zeros(2, 3, 2, 64, dtype=BF16, **new)
    table, i2 = torch.zeros(2, 2, dtype=torch.int32, **new), torch.zeros(2, dtype=torch.int32, **new)
    mask = torch.ones(2, 3, dtype=torch.int64, **new)
    write = lambda **o: ets.block_write(**{**dict(x=x, codes=codes, scales=scales, page_table=table, first=i2, counts=i2, page_size=8), **o})  # noqa: E731
    attend = lambda **o: ets.attend_blocks(**{**dict(q=x, k_codes=codes, k_scales=scales, v_codes=codes, v_scales=scales, page_table=table,  # noqa: E731
                                                     seq_lens=i2, page_size=8, L=16), **o})
    probs, uniform = torch.zeros(2, 3, 9, **new), torch.zeros(2, 3, **new)
    tokens = torch.zeros(2, 3, dtype=torch.int32, **new)
    verify = lambda **o: ets.verify_drafts(**{**dict(probs=probs, tokens=tokens, uniform=uniform), **o})  # noqa: E731
    refs = torch.zeros(4, dtype=torch.int32, **new)
    for error, call in [
        (ValueError, lambda: write(x=x.float().requires_grad_())),
        (TypeError, lambda: write(x=x.double())),
        (ValueError, lambda: write(x=x[:, :, :1])),
        (ValueError, lambda: write(x=x.transpose(2, 3))),
        (ValueError, lambda: write(scales=scales[:3])),
        (ValueError, lambda: write(scales=scales[:, :1])),
        (TypeError, lambda: write(scales=scales.int())),
        (TypeError, lambda: write(codes=codes.int())),
        (ValueError, lambda: write(codes=codes[:1].expand(16, 2, 64))),
        (ValueError, lambda: write(scales=scales[:1].expand(4, 2))),
        (ValueError, lambda: write(page_size=6)),
        (ValueError, lambda: write(page_size=0)),
        (ValueError, lambda: write(page_size=1 << 30)),
        (ValueError, lambda: write(page_table=table[:1])),
        (TypeError, lambda: write(page_table=table.long())),
        (TypeError, lambda: write(first=i2.long())),
        (ValueError, lambda: write(counts=i2[:1])),
        (ValueError, lambda: ets.block_keep(codes, scales, table, i2, torch.zeros(2, 65, dtype=torch.int32, **new), i2, 8)),
        (TypeError, lambda: ets.block_keep(codes, scales, table, i2, mask, i2, 8)),
        (TypeError, lambda: ets.block_keep(codes, scales, table, i2, None, i2, 8)),
        (ValueError, lambda: ets.block_keep(codes, scales, table, i2, tokens[:1], i2, 8)),
        (TypeError, lambda: attend(q=x.float())),
        (ValueError, lambda: attend(q=x.clone().requires_grad_())),
        (ValueError, lambda: attend(q=x[..., :32])),
        (ValueError, lambda: attend(q=x[:, :, :1])),
        (ValueError, lambda: attend(v_scales=scales.repeat_interleave(2, 0))),
        (ValueError, lambda: attend(L=17)),
        (ValueError, lambda: attend(L=-1)),
        (ValueError, lambda: attend(tree_mask=mask)),
        (ValueError, lambda: attend(tree_mask=mask[:, :2], first=i2)),
        (TypeError, lambda: attend(tree_mask=tokens, first=i2)),
        (ValueError, lambda: attend(first=i2[:1])),
        (ValueError, lambda: attend(k_codes=torch.zeros(16, 2, 288, dtype=torch.uint8, **new))),
        (ValueError, lambda: verify(probs=probs.clone().requires_grad_())),
        (TypeError, lambda: verify(probs=probs.double())),
        (ValueError, lambda: verify(probs=probs[..., :0])),
        (ValueError, lambda: verify(probs=torch.zeros(1, 65, 4, **new))),
        (ValueError, lambda: verify(tokens=tokens[:1])),
        (TypeError, lambda: verify(tokens=mask)),
        (TypeError, lambda: verify(uniform=uniform.double())),
        (ValueError, lambda: verify(draft_probs=probs)),
        (ValueError, lambda: verify(draft_probs=probs[:, :2].to(BF16))),
        (ValueError, lambda: verify(draft_probs=probs[:, :2], tree_mask=mask)),
        (TypeError, lambda: verify(tree_mask=tokens)),
        (ValueError, lambda: verify(lens=i2[:1])),
        (ValueError, lambda: verify(workspace=torch.zeros(8, dtype=torch.uint8, **new))),
        (TypeError, lambda: ets.pages_extend(refs.long(), table, i2, 8)),
        (ValueError, lambda: ets.pages_extend(refs, table, i2, 0)),
        (ValueError, lambda: ets.pages_extend(refs, table[:1].expand(2, 2), i2, 8)),
        (ValueError, lambda: ets.pages_extend(refs[::2], table, i2, 8)),
        (ValueError, lambda: ets.pages_free(refs, table, i2[:1], 8)),
        (ValueError, lambda: ets.pages_fork(refs, table, i2, 8, i2, [codes[:15]])),
        (ValueError, lambda: ets.pages_fork(refs, table, i2, 8, i2, [codes[:, :1]])),
        (ValueError, lambda: ets.pages_fork(refs, table, i2, 8, i2, out=table[:1])),
        (TypeError, lambda: ets.pages_fork(refs, table, i2, 8, i2, codes)),
        (TypeError, lambda: ets.pages_copy([codes] * 65, i2, i2, 4)),
        (ValueError, lambda: ets.pages_copy([codes], i2, i2[:1], 4)),
        (ValueError, lambda: ets.pages_copy([codes], i2, i2, -1)),
        (ValueError, lambda: ets.pages_compact(refs, table, [codes.cpu()])),
        (ValueError, lambda: ets.pages_compact(refs, table, [torch.zeros(4, 2, requires_grad=True, **new)])),
    ]:
        with pytest.raises(error):
            call()


def test_the_example():
    """examples/speculative_decode.py: graph replays follow the eager steps, attention is that of the cache, pages are counted."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_decode.py")
    loader = importlib.util.spec_from_file_location("speculative_decode", path)
    example = importlib.util.module_from_spec(loader)
    loader.loader.exec_module(example)

    def decoder():
        d = example.SpeculativeDecoder(2, 3, 200, pages=100, heads=4, kv_heads=2, dim=64, drafts=10, vocabulary=50, page=16, block=8)
        d.prefill(120, piece=48)
        d.project()
        return d

    a, b = decoder(), decoder()
    graph, held = a.capture()
    for _ in range(4):
        before, tree = b.lens.cpu(), b.tree.cpu()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        # b's cache as attention sees it: with the tree's rows, before the accepted ones move
        reach = b.lens + b.drafts
        ets.pages_extend(b.refs, b.table, reach, b.page)
        positions = b.lens[:, None] + b.depth
        b._write(b._turned(b.key, positions), b.value, b.table, b.lens, b.drafts)
        kc, ks, vc, vs = (t.view(torch.uint8).cpu() for t in b.pool)
        lists = spec.seen(b.table.cpu(), b.page, 100, reach.cpu(), b.capacity, 10, before, tree)
        want = spec.attend(b._turned(b.q, positions).cpu(), kc, ks, vc, vs, lists)
        out, new, counts, lacking = b.step()
        close(got[0], want[0], want[2], BF16)
        for x, y in zip(got, (out, new, counts, lacking)):
            assert torch.equal(x, y)
        for x, y in zip((a.refs, a.table, a.lens, a.tokens), (b.refs, b.table, b.lens, b.tokens)):
            assert torch.equal(x, y)
        for x, y in zip(a.pool, b.pool):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        table = a.table.cpu()
        assert torch.equal(a.refs.cpu(), torch.bincount(table[table >= 0].long(), minlength=100).int())
        a.project(), b.project()
    assert int(got[2].max()) > 1 and int(got[3].sum()) == 0
    a.finish()
    used = int((a.refs > 0).sum())
    assert used == int(((a.lens + 15) // 16).sum()) and (a.refs[:used] > 0).all() and int(a.table.max()) == used - 1
