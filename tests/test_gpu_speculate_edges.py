"""The operators of a speculative step at the edges of what their documentation allows."""
import pytest
import torch

import exact_top_selection_amd as ets
from tests import speculate_reference as spec
from tests.test_gpu_speculate import filled, ints, pages, run_blocks, same_codes, same_pages, tree
from tests.test_gpu_step import BF16, FP16, FP32, close, dev, gen
from tests.test_gpu_step_edges import close_where_numbers

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


# ---- more workgroups than a launch holds (2^32 lanes: 2^24 workgroups of 256 lanes, 2^26 of one wave)

def test_copies_of_more_pieces_than_a_launch_holds():
    n = (1 << 18) + 1
    held = torch.randint(0, 256, (64, 2 * n, 3), dtype=torch.uint8, device=dev())
    want = held.clone()
    order = torch.randperm(2 * n, device=dev()).int()
    src, dst = order[:n].contiguous(), order[n:].contiguous()
    want[:, dst.long()] = held[:, src.long()]
    ets.pages_copy(list(held.unbind(0)), src, dst, 2 * n)
    assert torch.equal(held, want)


def test_branches_of_more_pieces_than_a_launch_holds():
    n = (1 << 18) + 1
    held = torch.randint(0, 256, (64, n + 1, 5), dtype=torch.uint8, device=dev())
    refs = torch.zeros(n + 1, dtype=torch.int32, device=dev())
    refs[0] = 1
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device=dev()), torch.ones(1, dtype=torch.int32, device=dev())
    parents = torch.zeros(n, dtype=torch.int32, device=dev())
    rows, lacking = ets.pages_fork(refs, table, lens, 2, parents, list(held.unbind(0)))
    assert torch.equal(rows[:, 0], torch.arange(1, n + 1, dtype=torch.int32, device=dev())) and not lacking.any()
    assert (refs == 1).all() and torch.equal(held, held[:, :1].expand_as(held))
    # more branches than that, of full pages
    many = (1 << 24) + 5
    of = torch.full((many,), -1, dtype=torch.int32, device=dev())
    of[::2] = 0
    rows, lacking = ets.pages_fork(refs, table, lens, 1, of)
    assert torch.equal(rows[:, 0], of) and not lacking.any() and int(refs[0]) == 1 + (many + 1) // 2


def test_writes_of_more_blocks_than_a_launch_holds():
    # one wave a block: 2^26 and more of them
    T, H = (1 << 13) + 1, 1 << 13
    table = torch.randperm(129, device=dev()).int().view(1, 129)
    x = torch.randn(1, T, 1, 32, device=dev()).to(BF16)
    codes = torch.zeros(129 * 64, H, 32, dtype=torch.uint8, device=dev())
    scales = torch.zeros(129 * 64, H, dtype=torch.uint8, device=dev())
    one = codes[:, :1].clone(), scales[:, :1].clone()
    at, n = ints(0).to(dev()), ints(T).to(dev())
    ets.block_write(x.expand(1, T, H, 32), codes, scales, table, at, n, 64)
    ets.block_write(x, *one, table, at, n, 64)
    assert bool((codes.view(torch.int64) == one[0].view(torch.int64)).all()) and bool((scales == one[1]).all()) and bool(one[1].any())
    # four waves a block, most of them of sequences without rows
    B, T, H = (1 << 12) + 1, 1 << 14, 8
    x = torch.randn(1, T, H, 256, device=dev()).to(BF16)
    table = torch.full((B, 257), -1, dtype=torch.int32, device=dev())
    table[0], table[-1] = torch.randperm(514, device=dev()).int().view(2, 257)
    first, counts = torch.zeros(B, dtype=torch.int32, device=dev()), torch.zeros(B, dtype=torch.int32, device=dev())
    first[-1] = 45
    counts[::B - 1] = T
    got, want = ((torch.zeros(514 * 64, H, 256, dtype=torch.uint8, device=dev()), torch.zeros(514 * 2, H, dtype=torch.uint8, device=dev()))
                 for _ in range(2))
    ets.block_write(x.expand(B, T, H, 256), *got, table, first, counts, 64)
    ets.block_write(x.expand(2, T, H, 256), *want, table[::B - 1].contiguous(), first[::B - 1].contiguous(), counts[::B - 1].contiguous(), 64)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and int((got[1] > 0).sum()) == (512 + 513) * H


def test_moves_of_more_rows_than_a_launch_holds():
    B, H = (1 << 12) + 1, 1 << 12
    codes = torch.randint(0, 256, (2 * B, H, 32), dtype=torch.uint8, device=dev()) & 0xF7  # numbers all
    scales = torch.randint(100, 150, (2 * B, H), dtype=torch.uint8, device=dev())
    table = torch.randperm(B, device=dev()).int().view(B, 1)
    first, counts = torch.zeros(B, dtype=torch.int32, device=dev()), torch.ones(B, dtype=torch.int32, device=dev())
    path = torch.ones(B, 2, dtype=torch.int32, device=dev())
    want = codes.clone(), scales.clone()
    for b in range(0, B, 1000):
        part = slice(b, min(b + 1000, B))
        ets.block_keep(*want, table[part], first[part], path[part], counts[part], 2)
    assert not torch.equal(want[0][::2], codes[::2])
    ets.block_keep(codes, scales, table, first, path, counts, 2)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


def test_verification_of_more_sequences_than_a_launch_holds():
    B = (1 << 24) + 3
    pick = torch.randint(0, 2, (B, 1), device=dev())
    probs = torch.zeros(B, 1, 2, dtype=FP16, device=dev()).scatter_(2, pick[:, None], 1.0)
    tokens, path, counts = ets.verify_drafts(probs, torch.zeros(1, 1, dtype=torch.int32, device=dev()).expand(B, 1),
                                             torch.full((1, 1), 0.5, device=dev()).expand(B, 1))
    assert torch.equal(tokens, pick.int()) and not path.any() and (counts == 1).all()


def test_attention_of_more_lists_than_a_launch_holds():
    """Refused, in either cache's form; as many as a launch does hold are computed."""
    one, page = ints(1).to(dev()), torch.zeros(1, 1, dtype=torch.int32, device=dev())

    def heads(H):
        q = torch.zeros(1, 1, 1, 32, dtype=BF16, device=dev()).expand(1, 1, H, 32)
        codes = torch.randint(0, 127, (1, H, 32), dtype=torch.uint8, device=dev())
        return q, codes, torch.randint(120, 134, (1, H), dtype=torch.uint8, device=dev())

    for H in ((1 << 21) + 1, (1 << 22) + 1):  # odd numbers, so that a workgroup takes one
        q, codes, scales = heads(H)
        with pytest.raises(ets.EtsError):
            ets.attend_blocks(q, codes, scales, codes, scales, page, one, 1, 1)
        with pytest.raises(ets.EtsError):
            ets.attend_paged(q, codes, scales.view(1, H, 1), codes, scales.view(1, H, 1), page, one, 1, 1)
    q, codes, scales = heads((1 << 21) - 1)
    want = (codes.view(torch.float8_e4m3fn).float() * torch.exp2(scales.float() - 127)[..., None]).to(BF16).view(1, 1, -1, 32)
    out, lse = ets.attend_blocks(q, codes, scales, codes, scales, page, one, 1, 1)
    assert torch.equal(out, want) and not lse.any()
    out, lse = ets.attend_paged(q, codes, scales.view(1, -1, 1), codes, scales.view(1, -1, 1), page, one, 1, 1)
    assert torch.equal(out, want) and not lse.any()


# ---- branches written over rows of the table

@pytest.mark.parametrize("form", ["rows behind the parents", "every second row", "in place", "columns"])
def test_fork_into_the_table_itself(form):
    """All rows of parents are read before any is written."""
    g = gen(72)
    B, M, page = 40, 9, 4
    P = B * M * 2
    wide = torch.full((B, 2 * M), -1, dtype=torch.int32)
    wide[:, :M] = torch.randperm(P, generator=g)[:B * M].view(B, M).int()
    refs = torch.zeros(P, dtype=torch.int32)
    refs[wide[:, :M].flatten().long()] = 1
    lens = torch.randint(0, M * page + 1, (B,), generator=g, dtype=torch.int32)
    buffers = [torch.randint(0, 256, (P, 37), generator=g, dtype=torch.uint8)]
    read, write = {"rows behind the parents": (slice(None), slice(B // 2, B)), "every second row": (slice(None), slice(1, B, 2)),
                   "in place": (slice(None), slice(None)), "columns": (slice(None), slice(None))}[form]
    column = M if form == "columns" else 0
    n = len(range(*write.indices(B)))
    parents = torch.randint(0, B // 2 if form == "rows behind the parents" else B, (n,), generator=g, dtype=torch.int32)
    want = spec.fork(refs, wide[:, :M], lens, page, parents, M)
    there, got, on = wide.to(dev()), refs.to(dev()), [t.to(dev()) for t in buffers]
    rows = there[write, column:column + M]
    out, lacking = ets.pages_fork(got, there[read, :M], lens.to(dev()), page, parents.to(dev()), on, out=rows)
    expect = wide.clone()
    expect[write, column:column + M] = torch.tensor(want[1], dtype=torch.int32)
    assert out is rows and torch.equal(there.cpu(), expect) and got.tolist() == want[0] and lacking.tolist() == want[2]
    same_pages(on, buffers, want[3], P)


def test_fork_into_the_table_itself_in_a_graph():
    """Replays, with eager work between, follow the eager calls."""
    g = gen(73)
    B, M, page, P = 6, 5, 4, 400

    def state():
        h = gen(74)
        table = torch.randperm(P, generator=h)[:B * M].view(B, M).int()
        refs = torch.zeros(P, dtype=torch.int32)
        refs[table.flatten().long()] = 1
        return refs.to(dev()), table.to(dev()), torch.randint(0, 256, (P, 37), generator=h, dtype=torch.uint8).to(dev())

    lens, parents = torch.zeros(B, dtype=torch.int32, device=dev()), torch.zeros(B, dtype=torch.int32, device=dev())

    def step(refs, table, pages):
        return ets.pages_fork(refs, table, lens, page, parents, [pages], out=table)[1]

    step(*state())  # warm
    a, b = state(), state()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step(*a)
    for _ in range(5):
        lens.copy_(torch.randint(0, M * page + 1, (B,), generator=g, dtype=torch.int32))
        parents.copy_(torch.randint(0, B, (B,), generator=g, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        lacking = step(*b)
        assert torch.equal(kept, lacking) and all(torch.equal(x, y) for x, y in zip(a, b))
        torch.cuda.synchronize()


# ---- attention with eight waves a workgroup: filled groups of 256 rows of 65 to 128 channels, room for long lists, several
# turns of the device; and with four waves next to that

@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("waves,form,B,T,Hq,Hkv,D,Dv,room", [
    (8, "tree", 32, 64, 64, 16, 128, 128, 8192), (8, "tree", 35, 32, 128, 16, 32, 96, 8192), (8, "tree", 64, 64, 32, 8, 96, 64, 9000),
    (8, "causal", 32, 200, 32, 16, 128, 96, 8200), (8, "causal", 70, 256, 8, 8, 96, 96, 8192),
    (4, "tree", 64, 63, 40, 8, 64, 32, 8192), (4, "tree", 35, 50, 96, 16, 32, 96, 8192), (4, "tree", 32, 64, 64, 16, 128, 128, 154),
    (4, "tree", 35, 31, 128, 16, 32, 96, 8192),
    (4, "causal", 32, 130, 32, 16, 128, 96, 8192), (4, "causal", 70, 300, 8, 8, 64, 64, 390)])
@pytest.mark.parametrize("spoilt", [False, True])
def test_eight_waves(waves, form, B, T, Hq, Hkv, D, Dv, room, dtype, spoilt):
    """Trees, triangles and padding; rows that are no numbers among the drafts, in the last rows and behind the length."""
    G, L, page, block = Hq // Hkv, T + 90, 16, 8
    assert (waves == 8) == (64 < max(D, Dv) <= 128 and T * G >= 256 and 2 * -(-T * G // 256) == -(-T * G // 128)
                            and room >= 8192 and B * Hkv * -(-T * G // 256) >= 2 * ets.device_limits()[0])
    g = gen(75)
    table, P = pages(B, -(-L // page), 1, g)
    kc, ks = filled(P * page, Hkv, D, block, g)
    vc, vs = filled(P * page, Hkv, Dv, block, g)
    q = torch.randn(B, T, Hq, D, generator=g).to(dtype)
    lens = torch.randint(T, L + 1, (B,), generator=g, dtype=torch.int32)
    first = lens - T
    first[1] += T // 3  # its last tokens are padding
    lens[2], first[2] = T // 2, 0
    table = torch.nn.functional.pad(table, (0, -(-room // page) - table.shape[1]), value=-1)
    mask = tree(B, T, g) if form == "tree" else None
    some = {0, 1, 2, B // 2, B - 1}
    if spoilt:
        for b in some:
            at = lambda p: spec.place(table[b], page, P, p)  # noqa: E731,B023
            start, end = int(first[b]), int(lens[b])
            vc[at(min(start + T // 2, end - 1)), :, 3], vc[at(end - 1), Hkv - 1, Dv - 1] = 0x7F, 0xFF
            kc[at(max(start, end - 2)), 0, 0] = 0xFF
            for p in range(end, min(-(-L // page) * page, end + 40)):  # never written
                kc[at(p)], vc[at(p)] = 0x7F, 0xFF
    out, lse = run_blocks(q, kc, ks, vc, vs, table, lens, page, room, first, mask)
    tokens = sorted({0, 1, T // 4, T // 2 - 1, T // 2, T - 2, T - 1})
    numbers = 0
    for b in some:
        for h in {0, Hkv - 1}:
            lists = spec.seen(table[b:b + 1], page, P, lens[b:b + 1], room, T, first[b:b + 1], None if mask is None else mask[b:b + 1])
            heads = slice(h * G, h * G + G)
            want = spec.attend(q[b:b + 1, tokens, heads], kc[:, h:h + 1], ks[:, h:h + 1], vc[:, h:h + 1], vs[:, h:h + 1],
                               [[lists[0][t] for t in tokens]])
            close_where_numbers(out[b:b + 1, tokens, heads], want[0], want[2], dtype)
            close_where_numbers(lse[b:b + 1, tokens, heads], want[1], want[3], FP32)
            numbers += int(torch.isnan(want[0]).any())
    assert (numbers > 0) == spoilt
    again = run_blocks(q, kc, ks, vc, vs, table, lens, page, room, first, mask)
    assert torch.equal(out.view(torch.uint8), again[0].view(torch.uint8)) and torch.equal(lse.view(torch.uint8), again[1].view(torch.uint8))


# ---- numbers that the documentation allows and that no program above brings

ENDS = [-0x80000000, -0x7FFFFFFF, -1, 0x7FFFFFFF, 0x7FFFFF00]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,Hq,Hkv,D,Dv,form", [(3, 4, 2, 64, 64, "causal"), (9, 2, 2, 128, 96, "tree"), (40, 6, 2, 96, 128, "causal"), (64, 2, 1, 128, 128, "tree"),
                                                (17, 12, 1, 256, 192, "tree"), (150, 2, 1, 64, 32, "causal"), (20, 5, 1, 160, 224, "causal")])
def test_attend_blocks_of_any_first_length_and_mask(T, Hq, Hkv, D, Dv, form, dtype):
    """Tokens that stand anywhere next to the length, bits of any kind, pages that are not there, a cache that is not whole pages."""
    g = gen(76)
    B, block, page, L = 24, 4, 12, 170
    table, P = pages(B, -(-L // page), 3, g)
    table[torch.rand(table.shape, generator=g) < 0.1] = -1
    table[3, :], table[4, 2] = P, P - 1
    S = P * page - block  # the last page is not whole: not there
    kc, ks = filled(P * page, Hkv, D, block, g)
    vc, vs = filled(P * page, Hkv, Dv, block, g)
    kc, vc, ks, vs = kc[:S], vc[:S], ks[:S // block], vs[:S // block]
    q = torch.randn(B, T, Hq, D, generator=g).to(dtype)
    lens = torch.randint(-3, L + 30, (B,), generator=g, dtype=torch.int32)
    first = (torch.rand(B, generator=g) * (L + T + 20) - T - 10).to(torch.int32)
    first[:5], lens[5:10] = ints(*ENDS), ints(*ENDS)
    first[10:12], lens[10:12] = 0, L
    mask = None
    if form == "tree":
        mask = torch.randint(-(1 << 63), (1 << 63) - 1, (B, T), generator=g)
        mask[::3] &= torch.randint(-(1 << 63), (1 << 63) - 1, (len(range(0, B, 3)), T), generator=g) & 0x1111111111111111
        mask[11], mask[12, ::2] = 0, 0
    out, lse = run_blocks(q, kc, ks, vc, vs, table, lens, page, L, first, mask)
    lists = spec.seen(table, page, S // page, lens, L, T, first, mask)
    want = spec.attend(q, kc, ks, vc, vs, lists)
    close(out, want[0], want[2], dtype)
    close(lse, want[1], want[3], FP32)
    nothing = torch.tensor([[not bool((row >= 0).any()) for row in rows] for rows in lists])
    assert nothing.any() and not nothing.all()
    assert not out.cpu()[nothing].any() and bool((lse.cpu()[nothing] == -float("inf")).all())


@pytest.mark.parametrize("block,page,D", [(4, 12, 64), (1, 3, 32), (20, 20, 256)])
def test_writes_at_the_ends_of_a_table(block, page, D):
    """Rows that stand across either end of the table, or beyond it; a cache that is not whole pages."""
    g = gen(77)
    B, T, H, M = 30, 25, 2, 4
    table, P = pages(B, M, 1, g)
    table[7, 3] = P - 1
    codes, scales = filled(P * page, H, D, block, g)
    S = (P - 1) * page + page // 2 // block * block
    codes, scales = codes[:S], scales[:S // block]
    first = torch.randint(M * page - T, M * page + 3, (B,), generator=g, dtype=torch.int32).clamp(min=0)
    first[:5], first[5] = ints(*ENDS), 0
    counts = torch.randint(-2, T + 3, (B,), generator=g, dtype=torch.int32)
    counts[10:15] = ints(*ENDS)
    x = torch.randn(B, T, H, D, generator=g).to(BF16)
    want = spec.block_write(x, codes, scales, table, first, counts, page)
    got = codes.to(dev()), scales.to(dev())
    ets.block_write(x.to(dev()), *got, table.to(dev()), first.to(dev()), counts.to(dev()), page)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])
    path = torch.stack([torch.randperm(T, generator=g) for _ in range(B)]).to(torch.int32)
    path[3, 2], path[9, 1], path[8, :3] = -0x80000000, 0x7FFFFFFF, ints(0, 1, 2)
    codes, scales = want
    want = spec.block_keep(codes, scales, table, first, path, counts, page)
    ets.block_keep(*got, table.to(dev()), first.to(dev()), path.to(dev()), counts.to(dev()), page)
    assert same_codes(got[0], want[0]) and torch.equal(got[1].cpu(), want[1])


def test_pages_of_any_numbers():
    g = gen(78)
    P, B, M, page = 300, 12, 9, 5
    held = [torch.randint(0, 256, (P, 21), generator=g, dtype=torch.uint8)]
    for turn in range(4):
        refs = torch.randint(-1, 2, (P,), generator=g, dtype=torch.int32)
        refs[:3] = ints(-0x80000000, -5, 0)
        table = torch.full((B, M), -1, dtype=torch.int32)
        used = (refs > 0).nonzero()[:, 0].int()
        some = torch.rand(B, M, generator=g) < 0.5
        table[some] = used[torch.randperm(used.numel(), generator=g)[:int(some.sum())]]
        table[1, 2], table[2, 0], table[3, 1] = 0x7FFFFFFF, -0x80000000, P
        lens = torch.randint(-3, M * page + 9, (B,), generator=g, dtype=torch.int32)
        lens[:5] = ints(*ENDS)
        parents = torch.randint(-2, B + 2, (15,), generator=g, dtype=torch.int32)
        parents[:2], parents[3:8] = ints(0x7FFFFFFF, -0x80000000), ints(0, 1, 2, 3, 4)
        got, on = refs.to(dev()), [t.to(dev()) for t in held]
        want = spec.fork(refs, table, lens, page, parents, M)
        rows, lacking = ets.pages_fork(got, table.to(dev()), lens.to(dev()), page, parents.to(dev()), on)
        assert got.tolist() == want[0] and rows.tolist() == want[1] and lacking.tolist() == want[2]
        same_pages(on, held, want[3], P)
        got, rows = refs.to(dev()), table.to(dev())
        want = spec.extend(refs, table, lens, page)
        lacking = ets.pages_extend(got, rows, lens.to(dev()), page)
        assert got.tolist() == want[0] and rows.tolist() == want[1] and lacking.tolist() == want[2]
        got, rows = refs.to(dev()), table.to(dev())
        want = spec.release(refs, table, lens, page)
        ets.pages_free(got, rows, lens.to(dev()), page)
        assert got.tolist() == want[0] and rows.tolist() == want[1]
    # branches of no table at all
    rows, lacking = ets.pages_fork(got, rows[:0], lens[:0].to(dev()), page, parents.to(dev()))
    assert rows.shape == (15, M) and bool((rows == -1).all()) and not lacking.any()


def test_verification_of_any_masks_and_lengths():
    g = gen(79)
    B, T, V = 50, 64, 40
    probs = torch.softmax(torch.randn(B, T, V, generator=g), -1)
    mask = torch.randint(-(1 << 63), (1 << 63) - 1, (B, T), generator=g)
    mask[::2] = tree(len(range(0, B, 2)), T, g)
    tokens = torch.randint(-2, V + 2, (B, T), generator=g, dtype=torch.int32)
    tokens[0, 1:6], tokens[1, :] = ints(*ENDS), 7
    lens = torch.randint(-2, T + 5, (B,), generator=g, dtype=torch.int32)
    lens[5:10] = ints(*ENDS)
    uniform = torch.rand(B, T, generator=g) * 0.2
    for m in (mask, None):
        want = spec.verify(probs, tokens, uniform, None, m, lens)
        got = ets.verify_drafts(probs.to(dev()), tokens.to(dev()), uniform.to(dev()), tree_mask=None if m is None else m.to(dev()), lens=lens.to(dev()))
        for a, b in zip(got, want):
            assert torch.equal(a.cpu(), b)
