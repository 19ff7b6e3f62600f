"""The decode operators on the GPU against the plain 64-bit forms of tests/decode_reference.py.

Run after test_gpu_dispatch.py (by its name): that file's check that workgroup i runs on XCD i % X holds in a process
whose launches so far leave the dealing at XCD 0, which grids of any size do not.
"""
import math

import pytest
import torch

import exact_top_selection_amd as ets
from tests import decode_reference as ref

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def dev():
    return torch.device("cuda:0")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def close(got, want, bound, dtype):
    """|got - want| <= bound + the rounding to the output's type, element by element; infinities equal."""
    got = got.cpu().double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want))
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine], want[~fine])
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    limit = bound + (want.abs() + bound) * ref.half_step(dtype) + tiny
    over = ((got - want).abs() - limit)[fine]
    assert not over.numel() or over.max() <= 0, "worst %g over its bound" % over.max()


def cache(S, H, D, g, size=1.0):
    """A cache of normal rows of differing size: (codes float8, scales, the same on the GPU)."""
    x = torch.randn(S, H, D, generator=g) * torch.exp(torch.randn(S, H, 1, generator=g)) * size
    codes, scales = ref.quantise(x)
    codes = codes.view(torch.float8_e4m3fn)
    return codes, scales, codes.to(dev()), scales.to(dev())


# ---- rope

ROPE = [  # N, H, D, R, offset, layout, scale, inverse
    (1, 128, 576, 64, 512, "interleaved", 1.0, False),
    (5, 3, 128, 128, 0, "half", 1.3, False),
    (33, 2, 96, 64, 16, "interleaved", 1.0, True),
    (7, 9, 64, 32, 8, "half", 0.5, True),
    (9, 2, 64, 30, 5, "half", 1.0, False),          # odd number of pairs, odd offset
    (9, 2, 64, 30, 5, "interleaved", 1.0, False),   # pairs across vectors
    (4, 1, 33, 20, 13, "half", 1.0, True),          # rows that are no whole vectors
    (3, 5, 7, 6, 1, "interleaved", 1.0, False),
    (2, 1, 1, 0, 0, "half", 1.0, False),            # nothing turns
    (2, 2, 4096, 4096, 0, "half", 1.0, False),
    (2, 2, 4095, 4094, 1, "interleaved", 1.0, False),
    (300, 1, 32, 2, 30, "interleaved", 1.0, False),
    (0, 4, 64, 64, 0, "half", 1.0, False),
]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("case", ROPE)
def test_rope(case, dtype):
    N, H, D, R, offset, layout, scale, inverse = case
    g = gen(1)
    x = torch.randn(N, H, D, generator=g).to(dtype)
    pos = torch.randint(-5, 1 << 20, (N,), generator=g, dtype=torch.int32)
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / max(R, 1))
    want, bound = ref.rope(x, pos, freq, layout, offset, scale, inverse)
    got = ets.rope(x.to(dev()), pos.to(dev()), freq.to(dev()), layout=layout, offset=offset, scale=scale, inverse=inverse)
    close(got, want, bound, dtype)
    rest = [d for d in range(D) if not offset <= d < offset + R]
    assert torch.equal(got.cpu()[..., rest], x[..., rest])


@pytest.mark.parametrize("layout,offset,R", [("half", 0, 64), ("interleaved", 8, 48), ("half", 3, 42)])
def test_rope_strides_and_in_place(layout, offset, R):
    g = gen(2)
    wide = torch.randn(70, 6, 101, generator=g).to(BF16).to(dev())
    x = wide[::2, 1:4, 5:69]  # strided rows that begin off a vector's boundary
    pos = torch.arange(35, dtype=torch.int32, device=dev())
    freq = 100.0 ** (-torch.arange(R // 2, dtype=torch.float64) / R).to(dev())
    plain = ets.rope(x.contiguous(), pos, freq, layout=layout, offset=offset)
    assert torch.equal(ets.rope(x, pos, freq, layout=layout, offset=offset), plain)
    before = wide.clone()
    assert ets.rope(x, pos, freq, layout=layout, offset=offset, out=x) is x
    assert torch.equal(x, plain)
    wide[::2, 1:4, 5:69] = before[::2, 1:4, 5:69]
    assert torch.equal(wide, before)  # nothing beside the rows was written


@pytest.mark.parametrize("layout,offset,R", [("half", 0, 32), ("interleaved", 4, 24), ("half", 1, 30)])
def test_rope_gradient(layout, offset, R):
    g = gen(3)
    N, H, D = 11, 3, 40
    pos = torch.randint(0, 1000, (N,), generator=g, dtype=torch.int32).to(dev())
    freq = (50.0 ** (-torch.arange(R // 2, dtype=torch.float64) / R)).to(dev())
    up = torch.randn(N, H, D, generator=g).to(dev())
    grad = ets.rope(up, pos, freq, layout=layout, offset=offset, scale=1.5, inverse=True)
    want, bound = ref.rope(up.cpu(), pos.cpu(), freq.cpu(), layout, offset, 1.5, True)
    close(grad, want, bound, FP32)
    # differences: the map is linear, so a step along a direction moves it by the map of the direction
    step = torch.randn(N, H, D, generator=g)
    moved = ref.rope(step, pos.cpu(), freq.cpu(), layout, offset, 1.5, False)[0]
    a, b = (moved * up.cpu().double()).sum(), (grad.cpu().double() * step.double()).sum()
    assert abs(a - b) <= (bound * step.abs().double()).sum() + want.abs().mul(step.abs()).sum() * ref.U32


# ---- the cache

@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("N,H,D,S", [(1, 1, 32, 1), (64, 1, 576, 300), (37, 3, 160, 50), (5, 8, 128, 9), (0, 1, 32, 4)])
def test_cache_write_and_read(N, H, D, S, dtype):
    g = gen(5)
    x = torch.randn(N, H, D, generator=g) * torch.exp(3 * torch.randn(N, H, 1, generator=g))
    if N > 4:
        x[0] = 0
        x[1, 0, :32] = 448 * 2.0 ** -3   # the border between two scales
        x[2, 0, 3] = -0.0
        x[3] *= 1e-7 if dtype == FP16 else 1e-37
        x[4] = 1e30 if dtype != FP16 else 60000
    x = x.to(dtype)
    slots = torch.randperm(S, generator=g)[:N].to(torch.int32)
    if N > 6:
        slots[5], slots[6] = -1, S + 7
    before, scales_before = torch.randint(0, 256, (S, H, D), generator=g, dtype=torch.uint8), \
        torch.randint(1, 247, (S, H, D // 32), generator=g, dtype=torch.uint8)
    want, want_scales = before.clone(), scales_before.clone()
    kept = (slots >= 0) & (slots < S)
    if kept.any():
        c, s = ref.quantise(x[kept])
        want[slots[kept].long()], want_scales[slots[kept].long()] = c, s
    codes, scales = before.to(dev()), scales_before.to(dev())
    ets.cache_write(x.to(dev()), slots.to(dev()), codes.view(torch.float8_e4m3fn), scales)
    assert torch.equal(scales.cpu(), want_scales)
    assert torch.equal(codes.cpu(), want)

    got = ets.cache_read(codes.view(torch.float8_e4m3fn), scales, slots.to(dev()), dtype=dtype).cpu()
    full = torch.zeros(N, H, D, dtype=torch.float64)
    if kept.any():
        full[kept] = ref.values(want[slots[kept].long()], want_scales[slots[kept].long()])
    assert torch.equal(got, full.to(FP32).to(dtype))  # every code times its scale here is a 32-bit number


def test_cache_every_code_and_scale():
    """All 256 codes under all scale bytes that are written, in each type."""
    codes = torch.arange(256, dtype=torch.uint8).view(8, 1, 32).repeat(246, 1, 1)
    scales = torch.arange(1, 247, dtype=torch.uint8).repeat_interleave(8).view(-1, 1, 1)
    slots = torch.arange(len(codes), dtype=torch.int32)
    want = ref.values(codes, scales)
    for dtype in (FP32, BF16, FP16):
        got = ets.cache_read(codes.to(dev()), scales.to(dev()), slots.to(dev()), dtype=dtype).cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(0.0), want.to(FP32).to(dtype).nan_to_num(0.0))
    # and values of the format survive a write in 32 bits
    keep = (scales.view(-1) > 1 + 9) & (codes[:, 0].view(-1, 32).view(len(codes), 32) & 127).ne(127).all(1)
    x = want[keep].to(FP32)
    c2, s2 = torch.zeros(len(x), 1, 32, dtype=torch.uint8, device=dev()), torch.zeros(len(x), 1, 1, dtype=torch.uint8, device=dev())
    at = torch.arange(len(x), dtype=torch.int32, device=dev())
    ets.cache_write(x.to(dev()), at, c2.view(torch.float8_e4m3fn), s2)
    assert torch.equal(ets.cache_read(c2, s2, at, dtype=FP32).cpu(), x)


def test_cache_write_of_values_that_are_not_finite():
    x = torch.linspace(-3, 3, 32).view(1, 1, 32).clone()
    plain, byte = ref.quantise(x)
    x[0, 0, 4], x[0, 0, 9], x[0, 0, 20] = math.nan, math.inf, -math.inf
    codes, scales = torch.zeros(1, 1, 32, dtype=torch.uint8, device=dev()), torch.zeros(1, 1, 1, dtype=torch.uint8, device=dev())
    ets.cache_write(x.to(dev()), torch.zeros(1, dtype=torch.int32, device=dev()), codes, scales)
    assert torch.equal(scales.cpu(), byte)
    got = codes.cpu()[0, 0]
    assert got[4] & 127 == 127 and got[9] == 0x7E and got[20] == 0xFE
    others = [i for i in range(32) if i not in (4, 9, 20)]
    assert torch.equal(got[others], plain[0, 0, others])


def test_cache_strides_and_far_slots():
    """A cache whose slots lie further apart than 2^31 bytes in all, and rows at odd addresses."""
    S, H, D = 70000, 1, 64
    room = torch.empty(S * 40000 + 64, dtype=torch.uint8, device=dev())
    codes = room.as_strided((S, H, D), (40000, D, 1), 3)
    scales = torch.zeros(S, H, 2, dtype=torch.uint8, device=dev())
    g = gen(6)
    x = torch.randn(4, H, D, generator=g).to(BF16)
    slots = torch.tensor([0, 53687, 53688, S - 1], dtype=torch.int32, device=dev())
    ets.cache_write(x.to(dev()), slots, codes, scales)
    c, s = ref.quantise(x)
    assert torch.equal(codes[slots.long()].cpu(), c)
    assert torch.equal(ets.cache_read(codes, scales, slots).cpu(), ref.values(c, s).to(BF16))
    q = torch.randn(1, 1, 2, D, generator=g).to(BF16)
    out, lse = ets.attend_selected(q.to(dev()), codes, scales, codes, scales, slots.view(1, 1, 4))
    lists = [[torch.arange(4)]]
    want = ref.attend(q, c, s, c, s, lists)
    close(out, want[0], want[2], BF16)
    close(lse, want[1], want[3], FP32)
    w = torch.ones(1, 1, 2)
    got = ets.index_scores(q.to(dev()), w.to(dev()), codes, scales, slots.view(1, 4), torch.tensor([4], dtype=torch.int32, device=dev()), 1, 4)
    want, bound = ref.index_scores(q, w, c, s, torch.arange(4, dtype=torch.int32).view(1, 4), [4], 1, 4)
    close(got, want, bound, FP32)


# ---- scores

SCORES = [  # B, T, H, D, L, page, lens
    (1, 1, 1, 32, 1, 1, [1]),
    (3, 1, 64, 128, 500, 64, [500, 0, 257]),
    (2, 4, 32, 128, 1100, 16, [1100, 1025]),
    (2, 3, 5, 96, 130, 48, [129, 64]),
    (1, 13, 64, 128, 70, 100, [65]),        # more query tiles than fit at once
    (2, 2, 17, 256, 90, 1, [-3, 1000]),     # lengths outside the rows
    (1, 1, 128, 192, 300, 7, [299]),
    (1, 2, 128, 256, 65, 64, [65]),
]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("case", SCORES)
def test_index_scores(case, dtype):
    B, T, H, D, L, page, lens = case
    g = gen(7)
    per = -(-L // page)
    codes, scales, cg, sg = cache(B * per * page, 1, D, g)
    table = torch.randperm(B * per, generator=g).to(torch.int32).view(B, per)
    q = torch.randn(B, T, H, D, generator=g).to(dtype)
    w = torch.randn(B, T, H, generator=g)
    lens = torch.tensor(lens, dtype=torch.int32)
    want, bound = ref.index_scores(q, w, codes, scales, table, lens, page, L)
    wide = torch.full((B * T, L + 5), 7.0, device=dev())
    got = ets.index_scores(q.to(dev()), w.to(dev()), cg, sg, table.to(dev()), lens.to(dev()), page, L, out=wide[:, :L])
    close(got, want, bound, FP32)
    assert (wide[:, L:] == 7).all()
    again = ets.index_scores(q.to(dev()), w.to(dev()), cg, sg, table.to(dev()), lens.to(dev()), page, L)
    assert torch.equal(got, again)


def test_index_scores_bad_pages_and_not_a_number():
    g = gen(8)
    codes, scales, cg, sg = cache(40, 1, 64, g)
    table = torch.tensor([[1, -1, 3, 9, 2 ** 30]], dtype=torch.int32)  # pages of 10: 9 and 2^30 lie outside
    q, w = torch.randn(1, 1, 4, 64, generator=g).to(BF16), torch.rand(1, 1, 4, generator=g) + 0.5
    lens = torch.tensor([50], dtype=torch.int32)
    want, bound = ref.index_scores(q, w, codes, scales, table, lens, 10, 50)
    got = ets.index_scores(q.to(dev()), w.to(dev()), cg, sg, table.to(dev()), lens.to(dev()), 10, 50)
    close(got, want, bound, FP32)
    cg.view(torch.uint8)[33, 0, 5] = 0x7F  # a NaN in one key stays with that key
    got = ets.index_scores(q.to(dev()), w.to(dev()), cg, sg, table.to(dev()), lens.to(dev()), 10, 50).cpu()
    assert torch.isnan(got[0, 23]) and int(torch.isnan(got).sum()) == 1


def test_index_scores_of_extreme_blocks():
    """Blocks of very different scales in one row, near the ends of the format."""
    g = gen(9)
    x = torch.randn(64, 1, 128, generator=g)
    x[:, :, :32] *= 1e-30
    x[:, :, 32:64] *= 1e4
    x[:32, :, 64:] *= 1e-4
    codes, scales = ref.quantise(x)
    table, lens = torch.tensor([[0]], dtype=torch.int32), torch.tensor([64], dtype=torch.int32)
    for dtype in (BF16, FP16):
        q, w = torch.randn(1, 2, 8, 128, generator=g).to(dtype), torch.randn(1, 2, 8, generator=g)
        want, bound = ref.index_scores(q, w, codes, scales, table, lens, 64, 64)
        got = ets.index_scores(q.to(dev()), w.to(dev()), codes.to(dev()), scales.to(dev()), table.to(dev()), lens.to(dev()), 64, 64)
        close(got, want, bound, FP32)


# ---- attention

def tree(B, T, g):
    mask = torch.zeros(B, T, dtype=torch.int64)
    for b in range(B):
        for t in range(T):
            parent = int(torch.randint(-1, t, (1,), generator=g)) if t else -1
            bits = (1 << t) | (int(mask[b, parent]) if parent >= 0 else 0)
            mask[b, t] = bits - (1 << 64) if bits >= 1 << 63 else bits  # as int64
    return mask


ATTEND = [  # mode, B, T, Hq, Hkv, D, Dv, L or K, page, lens (paged), tree
    ("selected", 2, 1, 8, 1, 64, 64, 70, 0, None, False),
    ("selected", 1, 1, 128, 1, 576, 512, 100, 0, None, False),    # one latent head
    ("selected", 2, 2, 16, 1, 576, 512, 33, 0, None, True),
    ("selected", 1, 3, 40, 1, 576, 512, 300, 0, None, False),
    ("selected", 1, 7, 32, 8, 128, 128, 200, 0, None, True),
    ("selected", 1, 1, 3, 3, 32, 32, 1, 0, None, False),
    ("selected", 1, 1, 4, 2, 160, 96, 31, 0, None, False),
    ("selected", 1, 2, 64, 1, 256, 256, 65, 0, None, False),
    ("selected", 1, 2, 4, 1, 64, 64, 0, 0, None, True),           # no list, only the tree
    ("selected", 1, 1, 2, 1, 576, 576, 40, 0, None, False),
    ("selected", 1, 1, 2, 1, 320, 64, 40, 0, None, False),
    ("paged", 1, 1, 64, 8, 128, 128, 700, 16, [700], False),
    ("paged", 3, 1, 8, 2, 128, 128, 129, 64, [129, 0, 1], False),  # an empty sequence
    ("paged", 2, 5, 12, 2, 96, 64, 100, 48, [33, 100], True),
    ("paged", 2, 33, 4, 2, 64, 64, 40, 1, [31, 0], True),          # a tree over two tiles, one without a prefix
    ("paged", 1, 64, 1, 1, 32, 32, 5, 100, [5], True),
    ("paged", 1, 13, 64, 1, 576, 512, 64, 64, [64], True),
    ("paged", 2, 2, 32, 4, 256, 256, 65, 100, [-1, 1000], False),  # lengths outside the sequence
    ("paged", 1, 4, 64, 1, 160, 160, 90, 7, [77], False),
    ("paged", 1, 1, 16, 1, 256, 32, 2100, 64, [2099], False),
]


def attention_case(case, dtype, seed=10):
    mode, B, T, Hq, Hkv, D, Dv, n, page, lens, has_tree = case
    g = gen(seed)
    latent = D == 576 and Dv == 512
    per = -(-(n + T) // page) if mode == "paged" else 0
    S = B * per * page if mode == "paged" else max(2 * n, 8) + B * T
    kc, ks, kg, ksg = cache(S, Hkv, D, g)
    if latent:
        vc, vs, vg, vsg = kc[..., :Dv], ks[..., :Dv // 32], kg[..., :Dv], ksg[..., :Dv // 32]
    else:
        vc, vs, vg, vsg = cache(S, Hkv, Dv, g)
    q = torch.randn(B, T, Hq, D, generator=g).to(dtype)
    kw, lists = {}, []
    if mode == "paged":
        table = torch.randperm(B * per, generator=g).to(torch.int32).view(B, per)
        kw = dict(page_table=table.to(dev()), seq_lens=torch.tensor(lens, dtype=torch.int32).to(dev()), page_size=page, L=n)
        clip = [max(0, min(x, n)) for x in lens]
        lists = [[ref.slots_of(table[b], page, torch.arange(clip[b]))] * T for b in range(B)]
        tree_slots = torch.stack([ref.slots_of(table[b], page, clip[b] + torch.arange(T)) for b in range(B)]).to(torch.int32)
    else:
        slots = torch.full((B, T, n), -1, dtype=torch.int32)
        for b in range(B):
            for t in range(T):
                m = n if t == 0 else int(torch.randint(0, n + 1, (1,), generator=g))
                slots[b, t, :m] = torch.randperm(S - B * T, generator=g)[:m].to(torch.int32)
                if n > 8 and t == 1:
                    slots[b, t] = slots[b, t][torch.randperm(n, generator=g)]  # holes anywhere
        kw = dict(slots=slots.to(dev()))
        lists = [[slots[b, t] for t in range(T)] for b in range(B)]
        tree_slots = (S - B * T + torch.arange(B * T, dtype=torch.int32)).view(B, T)
    args = (None, None)
    if has_tree:
        mask = tree(B, T, g)
        args = (tree_slots, mask)
        kw.update(tree_slots=tree_slots.to(dev()), tree_mask=mask.to(dev()))
    want = ref.attend(q, kc, ks, vc, vs, lists, *args)
    fn = ets.attend_paged if mode == "paged" else ets.attend_selected
    return fn, q, (kg, ksg, vg, vsg), kw, want


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("case", ATTEND)
def test_attention(case, dtype):
    fn, q, caches, kw, want = attention_case(case, dtype)
    out, lse = fn(q.to(dev()), *caches, **kw)
    close(out, want[0], want[2], dtype)
    close(lse, want[1], want[3], FP32)
    out2, lse2 = fn(q.to(dev()), *caches, **kw)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("shape", [(64, 1, 128, 128), (16, 2, 64, 64), (128, 1, 576, 512), (8, 1, 320, 64)])
def test_attention_of_scores_far_apart(shape, order, dtype):
    """Sizes of keys over 2^12, so that scores pass each other by far more than a softmax reference lets them."""
    Hq, Hkv, D, Dv = shape
    g, n = gen(12), 500
    x = torch.randn(n, Hkv, D, generator=g, dtype=torch.float64) * 2.0 ** (12 * torch.arange(n).double() / n - 4).view(n, 1, 1)
    codes, scales = ref.quantise(x)
    vc, vs = ref.quantise(torch.randn(n, Hkv, Dv, generator=g, dtype=torch.float64))
    slots = {"rising": torch.arange(n), "falling": torch.arange(n).flip(0), "mixed": torch.randperm(n, generator=g)}[order]
    q = torch.randn(1, 1, Hq, D, generator=g).to(dtype)
    out, lse, eo, el = ref.attend(q, codes, scales, vc, vs, [[slots]])
    got, l = ets.attend_selected(q.to(dev()), codes.to(dev()), scales.to(dev()), vc.to(dev()), vs.to(dev()),
                                 slots.to(torch.int32).view(1, 1, n).to(dev()))
    close(got, out, eo, dtype)
    close(l, lse, el, FP32)


def test_attention_row_that_sees_nothing():
    """No valid slot, an empty tree line, and a slot outside the cache: out 0 and lse -inf, next to rows that see something."""
    g = gen(11)
    kc, ks, kg, ksg = cache(16, 1, 64, g)
    q = torch.randn(2, 2, 4, 64, generator=g).to(BF16).to(dev())
    slots = torch.full((2, 2, 40), -1, dtype=torch.int32, device=dev())
    slots[0, 0, 39] = 3
    slots[1, 0, 2], slots[1, 0, 5] = 16, 2 ** 31 - 1
    mask = torch.tensor([[0, 0], [0, 2]], device=dev())
    tree_slots = torch.tensor([[0, 1], [5, 6]], dtype=torch.int32, device=dev())
    out, lse = ets.attend_selected(q, kg, ksg, kg, ksg, slots, tree_slots=tree_slots, tree_mask=mask)
    for b, t in ((0, 1), (1, 0)):
        assert (out[b, t] == 0).all() and (lse[b, t] == -math.inf).all()
    one = ref.values(kc, ks).to(BF16)
    assert torch.equal(out[0, 0].cpu(), one[3].expand(4, -1)) and torch.equal(out[1, 1].cpu(), one[6].expand(4, -1))
    out, lse = ets.attend_paged(q, kg, ksg, kg, ksg, torch.zeros(2, 1, dtype=torch.int32, device=dev()),
                                torch.tensor([0, 1], dtype=torch.int32, device=dev()), 16, 16)
    assert (out[0] == 0).all() and (lse[0] == -math.inf).all() and torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("mode", ["selected", "paged"])
def test_attention_ignores_what_is_not_seen(mode):
    """Rows of NaN codes at every slot that no token sees, and extreme scores, change nothing."""
    g = gen(12)
    S, D, n = 128, 64, 40
    kc, ks, kg, ksg = cache(S, 1, D, g, 30.0)
    q = (torch.randn(1, 2, 4, D, generator=g) * 20).to(BF16)
    page, table = 8, torch.randperm(16, generator=g).to(torch.int32).view(1, 16)
    lens = torch.tensor([n], dtype=torch.int32)
    seen = ref.slots_of(table[0], page, torch.arange(n))
    want = ref.attend(q, kc, ks, kc, ks, [[seen, seen]])
    hidden = torch.ones(S, dtype=torch.bool)
    hidden[seen] = False
    kg.view(torch.uint8)[hidden.to(dev())] = 0x7F
    if mode == "paged":
        out, lse = ets.attend_paged(q.to(dev()), kg, ksg, kg, ksg, table.to(dev()), lens.to(dev()), page, 128)
    else:
        slots = torch.full((1, 2, 64), -1, dtype=torch.int32)
        slots[..., 10:50] = seen.to(torch.int32)
        hide = int(hidden.nonzero()[0])
        out, lse = ets.attend_selected(q.to(dev()), kg, ksg, kg, ksg, slots.to(dev()),
                                       tree_slots=torch.full((1, 2), hide, dtype=torch.int32, device=dev()),
                                       tree_mask=torch.zeros(1, 2, dtype=torch.int64, device=dev()))
    close(out, want[0], want[2], BF16)
    close(lse, want[1], want[3], FP32)


def test_attention_strides_streams_and_workspace():
    """Strided queries and caches, an own workspace, another stream: the same bits as the plain call."""
    g = gen(13)
    B, T, Hq, Hkv, D, n = 2, 3, 8, 2, 128, 600
    _, _, kg, ksg = cache(n, Hkv, D, g)
    q = torch.randn(B, T, Hq, D, generator=g).to(FP16).to(dev())
    slots = torch.randint(-1, n, (B, T, n), generator=g, dtype=torch.int32).to(dev())
    plain = ets.attend_selected(q, kg, ksg, kg, ksg, slots)
    q2 = torch.empty(T, Hq + 1, B, D + 3, dtype=FP16, device=dev())[:, 1:, :, 1:D + 1].permute(2, 0, 1, 3)
    q2.copy_(q)
    k2 = torch.zeros(Hkv, n, 2 * D + 5, dtype=torch.uint8, device=dev())[:, :, 5:D + 5].transpose(0, 1)
    k2.copy_(kg.view(torch.uint8))
    s2 = torch.zeros(n, 3, Hkv, D // 32, dtype=torch.uint8, device=dev())[:, 1]
    s2.copy_(ksg)
    wide = torch.zeros(T, B, n + 9, dtype=torch.int32, device=dev())[..., 4:n + 4].transpose(0, 1)
    wide.copy_(slots)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device=dev())
        out, lse = ets.attend_selected(q2, k2, s2, k2, s2, wide, workspace=ws)
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [64, 128, 192, 256, 576])
def test_scale_bytes_at_odd_addresses(D, dtype):
    """Rows of scale bytes that start anywhere, the last ending with its allocation's view: the same bits as aligned ones."""
    g = gen(14)
    n, blocks = 301, D // 32
    _, _, kg, ksg = cache(n, 1, D, g)
    odd = torch.zeros(n * (blocks + 3) + 1, dtype=torch.uint8, device=dev())[1:].view(n, 1, blocks + 3)[..., 3:]
    odd.copy_(ksg)
    q = torch.randn(2, 2, 6, D, generator=g).to(dtype).to(dev())
    slots = torch.randint(0, n, (2, 2, 77), generator=g, dtype=torch.int32).to(dev())
    slots[..., 0] = n - 1
    one, two = ets.attend_selected(q, kg, ksg, kg, ksg, slots), ets.attend_selected(q, kg, odd, kg, odd, slots)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    if D <= 256:
        w = torch.rand(2, 2, 6, generator=g).to(dev())
        table = torch.arange(n - 1, -1, -1, device=dev(), dtype=torch.int32).repeat(2, 1)
        lens = torch.tensor([n, 200], device=dev(), dtype=torch.int32)
        assert torch.equal(ets.index_scores(q, w, kg, ksg, table, lens, 1, n), ets.index_scores(q, w, kg, odd, table, lens, 1, n))


def test_the_operators_in_a_graph():
    """A decode step captured once; each replay, with new inputs and eager work between, equals the eager step."""
    g = gen(14)
    B, H, D, L, page, k = 3, 16, 128, 2000, 16, 64
    per = L // page
    _, _, kg, ksg = cache(B * per * page, 1, D, g)
    table = torch.randperm(B * per, generator=g).to(torch.int32).view(B, per).to(dev())
    lens = torch.tensor([2000, 70, 1], dtype=torch.int32, device=dev())
    x = torch.zeros(B, H, D, dtype=BF16, device=dev())
    w = torch.rand(B, 1, H, generator=g).to(dev())
    pos, freq = lens.clone(), torch.rand(32, dtype=torch.float64, device=dev())
    slots = torch.zeros(B, k, dtype=torch.int32, device=dev())

    def step():
        q = ets.rope(x, pos, freq, layout="half", offset=64)
        row = ets.index_scores(q[:, None], w, kg, ksg, table, lens, page, L)
        ets.topk_paged(row, lens, table, slots, page)
        a = ets.attend_selected(q[:, None], kg, ksg, kg, ksg, slots[:, None])
        b = ets.attend_paged(q[:, None], kg, ksg, kg, ksg, table, lens, page, L)
        return (q, row, *a, *b, ets.cache_read(kg, ksg, slots[:, 0].contiguous()))

    step()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            held = step()
    for rep in range(4):
        x.copy_(torch.randn(B, H, D, generator=g).to(BF16))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for i, (a, b) in enumerate(zip(got, step())):
            if i in (2, 3):  # the selection's order is free; with it the order of the sums
                torch.testing.assert_close(a, b, rtol=0.02, atol=0.02)
            elif i < 6:
                assert torch.equal(a, b), i
        torch.cuda.synchronize()


def test_refusals():
    g = gen(15)
    _, _, kg, ksg = cache(8, 2, 64, g)
    q = torch.zeros(2, 1, 4, 64, dtype=BF16, device=dev())
    slots = torch.zeros(2, 1, 3, dtype=torch.int32, device=dev())
    i2 = torch.zeros(2, dtype=torch.int32, device=dev())
    table = torch.zeros(2, 1, dtype=torch.int32, device=dev())
    x = torch.zeros(2, 2, 64, dtype=BF16, device=dev())
    freq = torch.zeros(4, dtype=torch.float64, device=dev())
    attend = lambda **o: ets.attend_selected(**{**dict(q=q, k_codes=kg, k_scales=ksg, v_codes=kg, v_scales=ksg, slots=slots), **o})  # noqa: E731
    for error, call in [
        (TypeError, lambda: attend(q=q.float())),
        (ValueError, lambda: attend(q=q[:, :, :3])),
        (ValueError, lambda: attend(q=q.transpose(2, 3))),
        (ValueError, lambda: attend(k_codes=kg[:4])),
        (ValueError, lambda: attend(k_scales=ksg[..., :1])),
        (TypeError, lambda: attend(k_codes=kg.view(torch.int8))),
        (ValueError, lambda: attend(v_codes=kg[:4], v_scales=ksg[:4])),
        (ValueError, lambda: attend(slots=slots[:1])),
        (TypeError, lambda: attend(slots=slots.long())),
        (ValueError, lambda: attend(tree_slots=slots[:, :, 0])),
        (ValueError, lambda: attend(tree_slots=slots[:, 0], tree_mask=torch.zeros(2, 1, dtype=torch.int64, device=dev()))),
        (ValueError, lambda: attend(q=q.clone().requires_grad_())),
        (ValueError, lambda: attend(q=torch.zeros(1, 1, 2, 640, dtype=BF16, device=dev()), slots=slots[:1],
                                    **dict(zip(("k_codes", "k_scales", "v_codes", "v_scales"), cache(4, 1, 640, g)[2:] * 2)))),
        (ValueError, lambda: ets.attend_paged(q, kg, ksg, kg, ksg, table, i2, 4, 5)),
        (ValueError, lambda: ets.attend_paged(q, kg, ksg, kg, ksg, table, i2, 0, 0)),
        (ValueError, lambda: ets.index_scores(q, torch.zeros(2, 1, 4, device=dev()), kg, ksg, table, i2, 4, 4)),
        (ValueError, lambda: ets.index_scores(q, torch.zeros(2, 1, 3, device=dev()), kg[:, :1], ksg[:, :1], table, i2, 4, 4)),
        (ValueError, lambda: ets.rope(x.float().requires_grad_(), i2, freq)),
        (ValueError, lambda: ets.rope(x, i2, freq, layout="other")),
        (ValueError, lambda: ets.rope(x, i2, freq, offset=60)),
        (TypeError, lambda: ets.rope(x, i2, freq.float())),
        (TypeError, lambda: ets.rope(x, i2.long(), freq)),
        (ValueError, lambda: ets.rope(x, i2, freq, out=x[:1].expand(2, 2, 64))),
        (ValueError, lambda: ets.cache_write(x, i2, kg[:, :1], ksg[:, :1])),
        (ValueError, lambda: ets.cache_write(x, i2, kg[:1].expand(8, 2, 64), ksg)),
        (ValueError, lambda: ets.cache_write(x.float().requires_grad_(), i2, kg, ksg)),
        (TypeError, lambda: ets.cache_read(kg, ksg, i2, dtype=torch.float64)),
        (ValueError, lambda: ets.cache_read(kg, ksg, i2, out=torch.zeros(2, 2, 32, dtype=BF16, device=dev()))),
    ]:
        with pytest.raises(error):
            call()


def test_the_example_step():
    """examples/sparse_decode.py: graph replays follow the eager steps, and the attention is that of the chosen slots."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "sparse_decode.py")
    spec = importlib.util.spec_from_file_location("sparse_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)

    def decoder():
        d = example.SparseDecoder(3, 300, 32, heads=16, index_heads=8, page=16)
        d.prefill(100)
        d.project()
        return d

    a, b = decoder(), decoder()
    graph, held = a.capture()
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        out, lse = held[0].clone(), held[1].clone()
        b.step()
        assert torch.equal(a.lens, b.lens) and int(a.lens[0]) == 101 + step
        assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8)) and torch.equal(a.index_scales, b.index_scales)
        assert torch.equal(a.scores, b.scores)
        assert torch.equal(a.chosen.sort(1).values, b.chosen.sort(1).values)
        # the slots chosen are those of the 32 highest scores
        top = a.scores[:, :300].topk(32, sorted=False).indices.cpu()
        slots = torch.stack([ref.slots_of(a.table.cpu()[i], 16, top[i]) for i in range(3)])
        assert torch.equal(a.chosen.cpu().long().sort(1).values, slots.sort(1).values)
        q = ets.rope(a.q, a.lens - 1, a.inv_freq, offset=example.LATENT).cpu()[:, None]
        kc, ks = a.codes.cpu(), a.scales.cpu()
        want = ref.attend(q, kc, ks, kc[..., :512], ks[..., :16], [[a.chosen.cpu()[i]] for i in range(3)])
        close(out[:, None], want[0], want[2], BF16)
        close(lse[:, None], want[1], want[3], FP32)
