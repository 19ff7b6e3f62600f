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


def close_where_numbers(got, want, bound, dtype):
    """close(), with numbers in the same places."""
    none = torch.isnan(want)
    assert torch.equal(torch.isnan(got.cpu()), none)
    close(got.cpu().masked_fill(none, 0), want.masked_fill(none, 0), bound.masked_fill(none, 0), dtype)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T", [5, 40])  # drafted tokens of one tile, and of two
@pytest.mark.parametrize("shape", [(2, 2, 64, 64), (12, 2, 128, 96), (4, 1, 192, 192), (3, 1, 256, 256), (6, 1, 256, 128),
                                   (3, 1, 320, 320), (2, 1, 576, 512)])
def test_drafted_tokens_that_are_no_numbers(shape, T, dtype):
    """A draft with a value that is no number spoils the channels and heads of the tokens that see it, and nothing else."""
    Hq, Hkv, D, Dv = shape
    g = gen(23)
    B, page, n = 2, 16, 70
    lens = torch.tensor([37, 70], dtype=torch.int32)
    per = -(-(n + T) // page)
    table = torch.randperm(B * per, generator=g).to(torch.int32).view(B, per)
    kc, ks, _, _ = cache(B * per * page, Hkv, D, g)
    latent = Dv == 512
    vc, vs = (kc[..., :Dv], ks[..., :Dv // 32]) if latent else cache(B * per * page, Hkv, Dv, g)[:2]
    drafts = torch.stack([ref.slots_of(table[b], page, int(lens[b]) + torch.arange(T)) for b in range(B)])
    # draft 0 is the root of all; 1 hangs on it, 2 on 1, the others on 0; nobody sees the last
    mask = torch.tensor([1, 3, 7] + [1 | 1 << t for t in range(3, T - 1)] + [1]).repeat(B, 1)
    codes = vc.view(torch.uint8)
    codes[drafts[0, 1], -1, 5], codes[drafts[1, 3], 0, Dv - 1] = 0x7F, 0xFF
    if not latent:
        kc.view(torch.uint8)[drafts[1, 2], 0, 0] = 0x7F
    codes[drafts[:, T - 1]], vs[drafts[:, T - 1]] = 0x7F, 255  # a place that was never written
    kc.view(torch.uint8)[drafts[:, T - 1]] = 0xFF
    q = torch.randn(B, T, Hq, D, generator=g).to(dtype)
    lists = [[ref.slots_of(table[b], page, torch.arange(int(lens[b])))] * T for b in range(B)]
    want = two_parts(q, kc, ks, vc, vs, lists, drafts, mask)
    assert torch.isnan(want[0][0, 1]).any() and torch.isfinite(want[0][:, 0]).all() and torch.isfinite(want[0][:, T - 1]).all()
    kg, ksg = kc.to(dev()), ks.to(dev())
    vg, vsg = (kg[..., :Dv], ksg[..., :Dv // 32]) if latent else (vc.to(dev()), vs.to(dev()))
    out, lse = ets.attend_paged(q.to(dev()), kg, ksg, vg, vsg, table.to(dev()), lens.to(dev()), page, n,
                                tree_slots=drafts.to(torch.int32).to(dev()), tree_mask=mask.to(dev()))
    close_where_numbers(out, want[0], want[2], dtype)
    close_where_numbers(lse, want[1], want[3], FP32)


def uneven_blocks(n, D, size, g):
    """A cache whose rows hold values of about `size`, blocks of zeros under scales of all sizes, and blocks whose codes are
    far smaller than their scale lets them be."""
    codes, scales = ref.quantise(torch.randn(n, 1, D, generator=g) * size)
    for block in range(D // 32):
        kind = torch.randint(0, 4, (n,), generator=g)
        at = slice(32 * block, 32 * block + 32)
        empty = kind == 1
        codes[empty, :, at] = 0
        scales[empty, :, block] = torch.tensor([1, 118, 246], dtype=torch.uint8)[torch.randint(0, 3, (int(empty.sum()), 1), generator=g)]
        small = kind == 2  # codes up to 2^-6, the same values as the others'
        codes[small, :, at] = torch.randint(0, 8, (int(small.sum()), 1, 32), generator=g, dtype=torch.uint8)
        scales[small, :, block] = (scales[small, :, block].int() + 14).clamp(max=246).to(torch.uint8)
    return codes, scales


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("size", [1.0, 1e-4, 1e-8, 1e-10, 1e-30])
def test_keys_with_blocks_of_zeros_and_small_codes(size, D, dtype):
    g = gen(24)
    n = 150
    kc, ks = uneven_blocks(n, D, size, g)
    kg, ksg = kc.to(dev()), ks.to(dev())
    q, w = torch.randn(1, 2, 8, D, generator=g).to(dtype), torch.randn(1, 2, 8, generator=g)
    table, lens = torch.arange(n, dtype=torch.int32).view(1, n), torch.tensor([n], dtype=torch.int32)
    want, bound = ref.index_scores(q, w, kc, ks, table, lens, 1, n)
    got = ets.index_scores(q.to(dev()), w.to(dev()), kg, ksg, table.to(dev()), lens.to(dev()), 1, n)
    close(got, want, bound, FP32)
    vc, vs, vg, vsg = cache(n, 1, D, g)
    q = (q.double() / size).clamp(-60000, 60000).to(dtype)  # scores of about 1, as far as the type goes
    want = two_parts(q, kc, ks, vc, vs, [[table[0], table[0]]])
    out, lse = ets.attend_paged(q.to(dev()), kg, ksg, vg, vsg, table.to(dev()), lens.to(dev()), 1, n)
    close(out, want[0], want[2], dtype)
    close(lse, want[1], want[3], FP32)


def test_sizes_are_not_cut_to_32_bits():
    new = dict(device="cuda:0")
    codes, scales = torch.zeros(8, 1, 64, dtype=torch.uint8, **new), torch.full((8, 1, 2), 127, dtype=torch.uint8, **new)
    q, w = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, **new), torch.zeros(1, 1, 4, **new)
    lens = torch.ones(1, dtype=torch.int32, **new)
    table = torch.zeros(1, 3, dtype=torch.int32, **new)
    for page, L in (((1 << 32) + 4, 4), (1 << 31, 4), (1 << 31, (1 << 32) + 4), (1 << 30, 0x7FFFF001)):
        with pytest.raises(ValueError, match="page_size must be"):
            ets.attend_paged(q, codes, scales, codes, scales, table, lens, page, L)
        with pytest.raises(ValueError, match="page_size must be"):
            ets.index_scores(q, w, codes, scales, table, lens, page, L)
    many = q[:, :, :1].expand(1, (1 << 32) + 1, 1, 64)  # one token's memory
    with pytest.raises(ValueError, match="tokens"):
        ets.index_scores(many, w[:, :, :1].expand(1, (1 << 32) + 1, 1), codes, scales, table, lens, 4, 0)
    with pytest.raises(ValueError, match="rows"):
        ets.attend_paged(many, codes, scales, codes, scales, table, lens, 4, 4)
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16, **new).expand(1, (1 << 32) + 1, 64)
    with pytest.raises(ValueError, match="heads"):
        ets.rope(x, lens, torch.zeros(2, dtype=torch.float64, **new), out=x)


def every_list(q, kc, ks, vc, vs, slots, sample, **kw):
    """attend_selected of all rows, with the oracle's results for the sampled sequences: (out, lse, want)."""
    kg, ksg = kc.to(dev()), ks.to(dev())
    vg, vsg = (kg[..., :vc.shape[2]], ksg[..., :vs.shape[2]]) if vc.data_ptr() == kc.data_ptr() else (vc.to(dev()), vs.to(dev()))
    out, lse = ets.attend_selected(q.to(dev()), kg, ksg, vg, vsg, slots.to(dev()), **kw)
    want = two_parts(q[sample], kc, ks, vc, vs, [[slots[b, t] for t in range(q.shape[1])] for b in sample])
    return out[sample], lse[sample], want


@pytest.mark.parametrize("size", [2.0 ** 112, 1.0, 2.0 ** -90])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("shape", [(600, 1, 64, 64), (600, 20, 128, 128), (600, 20, 256, 256), (300, 4, 576, 512), (300, 64, 576, 512),
                                   (300, 2, 320, 320)])
def test_values_near_the_ends_of_the_range(shape, order, size):
    """Many lists, so that a wave takes several tiles: scores pass each other by up to 2^20, values reach 2^115 and 2^-90."""
    B, Hq, D, Dv = shape
    g, n = gen(25), 400
    x = torch.randn(n, 1, D, generator=g, dtype=torch.float64) * size
    x[..., D - 32:] = 0
    x[..., D - 1] = 20 * torch.arange(n).double().view(n, 1) / n / math.log2(math.e) * math.sqrt(D)  # the score of a query's last channel
    kc, ks = ref.quantise(x)
    vc, vs = (kc[..., :Dv], ks[..., :Dv // 32]) if Dv == 512 else ref.quantise(x[..., torch.arange(Dv) % (D - 32)])
    q = torch.zeros(B, 1, Hq, D, dtype=BF16)
    q[..., D - 1] = (torch.arange(B * Hq).view(B, 1, Hq) % 5 - 2) / 2
    slots = {"rising": torch.arange(n), "falling": torch.arange(n).flip(0), "mixed": torch.randperm(n, generator=g)}[order]
    out, lse, want = every_list(q, kc, ks, vc, vs, slots.to(torch.int32).expand(B, 1, n).contiguous(), [0, B // 2, B - 1])
    close(out, want[0], want[2], BF16)
    close(lse, want[1], want[3], FP32)


@pytest.mark.parametrize("behind", [True, False])
@pytest.mark.parametrize("shape", [(16, 64, 64), (32, 128, 128), (16, 256, 256), (64, 576, 512), (32, 320, 320)])
def test_scores_of_minus_infinity(shape, behind):
    """Keys whose score leaves the 32-bit range: alone in a list they are nothing, before others they weigh nothing."""
    Hq, D, Dv = shape
    g, n = gen(26), 200
    x = torch.zeros(n, 1, D, dtype=torch.float64)
    x[..., :D - 32] = torch.randn(n, 1, D - 32, generator=g)
    x[..., D - 1] = 8.0
    if behind:
        x[160:, 0, D - 1] = 2.0 ** -126 * (torch.arange(40) % 5).double()
    kc, ks = ref.quantise(x)
    vc, vs = (kc[..., :Dv], ks[..., :Dv // 32]) if Dv == 512 else ref.quantise(torch.randn(n, 1, Dv, generator=g).double())
    q = torch.zeros(300, 1, Hq, D, dtype=BF16)
    q[..., D - 1] = -2.0 ** 127
    slots = torch.arange(n, dtype=torch.int32).expand(300, 1, n).contiguous()
    kg, ksg = kc.to(dev()), ks.to(dev())
    vg, vsg = (kg[..., :Dv], ksg[..., :Dv // 32]) if Dv == 512 else (vc.to(dev()), vs.to(dev()))
    out, lse = ets.attend_selected(q.to(dev()), kg, ksg, vg, vsg, slots.to(dev()))
    want = two_parts(q[:1], kc, ks, vc, vs, [[torch.arange(160, n) if behind else torch.arange(0)]])
    for b in (0, 299):
        close(out[b:b + 1], want[0], want[2], BF16)
        close(lse[b:b + 1], want[1], want[3], FP32)


def test_derivatives_are_refused_not_dropped():
    """Inputs and outputs that require gradients, and inputs that carry a tangent."""
    import torch.autograd.forward_ad as forward
    g = gen(27)
    _, _, kg, ksg = cache(8, 1, 64, g)
    q = torch.randn(1, 1, 4, 64, generator=g).to(BF16).to(dev())
    x = torch.randn(2, 1, 64, generator=g).to(dev())
    w, i2 = torch.ones(1, 1, 4, device=dev()), torch.arange(2, dtype=torch.int32, device=dev())
    freq = torch.ones(8, dtype=torch.float64, device=dev())
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device=dev()), torch.ones(1, dtype=torch.int32, device=dev())
    slots = torch.zeros(1, 1, 3, dtype=torch.int32, device=dev())
    calls = [(x, lambda t: ets.rope(t, i2, freq)), (freq, lambda t: ets.rope(x, i2, t)), (x, lambda t: ets.cache_write(t, i2, kg, ksg)),
             (q, lambda t: ets.index_scores(t, w, kg, ksg, table, lens, 4, 4)),
             (w, lambda t: ets.index_scores(q, t, kg, ksg, table, lens, 4, 4)),
             (q, lambda t: ets.attend_selected(t, kg, ksg, kg, ksg, slots)),
             (q, lambda t: ets.attend_paged(t, kg, ksg, kg, ksg, table, lens, 4, 4))]
    outs = [lambda: ets.rope(x, i2, freq, out=torch.zeros_like(x, requires_grad=True)),
            lambda: ets.index_scores(q, w, kg, ksg, table, lens, 4, 4, out=torch.zeros(1, 4, device=dev(), requires_grad=True)),
            lambda: ets.cache_read(kg, ksg, i2, out=torch.zeros(2, 1, 64, dtype=BF16, device=dev(), requires_grad=True))]
    for t, call in calls:
        call(t)
        with pytest.raises(ValueError, match="gradient"):
            call(t.clone().requires_grad_())
        with torch.no_grad():
            call(t.clone().requires_grad_())
        with forward.dual_level():
            call(t)
            with pytest.raises(ValueError, match="forward-mode"):
                call(forward.make_dual(t, torch.ones_like(t)))
    for call in outs:
        with pytest.raises(ValueError, match="gradient"):
            call()


@pytest.mark.parametrize("layout,offset,R", [("half", 0, 64), ("interleaved", 8, 48), ("half", 3, 42), ("interleaved", 1, 62)])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("span", [64, 1 << 20, (1 << 31) - 1])
def test_rope_coefficients_are_rounded_once(span, inverse, layout, offset, R):
    """Cosine and sine times the scale within half a step of 32 bits, at positions near and far."""
    g = gen(28)
    N, H, D, scale = 500, 2, 64, 1.3
    x = torch.randn(N, H, D, generator=g)
    pos = torch.randint(-span, span, (N,), generator=g).to(torch.int32)
    freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)
    want, _ = ref.rope(x, pos, freq, layout, offset, scale, inverse)
    # two coefficients, two products, each off by half a step of its size; the series beneath 2^-36
    i = torch.arange(R // 2)
    ia, ib = (offset + 2 * i, offset + 2 * i + 1) if layout == "interleaved" else (offset + i, offset + R // 2 + i)
    angle = pos.double()[:, None, None] * freq
    c, s = angle.cos().abs() * scale, angle.sin().abs() * scale
    a, b = x.double().abs()[..., ia], x.double().abs()[..., ib]
    bound = torch.zeros_like(want)
    bound[..., ia], bound[..., ib] = a * c + b * s, b * c + a * s
    bound = bound * 2 * ref.U32 * (1 + ref.U32) + bound.amax(-1, keepdim=True) * 2.0 ** -36
    got = ets.rope(x.to(dev()), pos.to(dev()), freq.to(dev()), layout=layout, offset=offset, scale=scale, inverse=inverse)
    close(got, want, bound, FP32)


@pytest.mark.parametrize("shape", [(16, 64, 64), (64, 128, 128), (8, 256, 256), (64, 576, 512), (16, 576, 512), (8, 320, 320)])
def test_log_sum_exp_of_one_key(shape):
    """It is the score itself: a product of one channel, its scaling, and the way through the exponential and back."""
    Hq, D, Dv = shape
    g, n = gen(29), 200
    kc, ks, kg, ksg = cache(n, 1, D, g)
    vc, vs, vg, vsg = (kc[..., :Dv], ks[..., :Dv // 32], kg[..., :Dv], ksg[..., :Dv // 32]) if Dv == 512 else cache(n, 1, Dv, g)
    q = torch.zeros(n, 1, Hq, D, dtype=BF16)
    q[..., 7] = (torch.randn(n, 1, Hq, generator=g) * 0.05).to(BF16)
    slots = torch.arange(n, dtype=torch.int32).view(n, 1, 1)
    _, lse = ets.attend_selected(q.to(dev()), kg, ksg, vg, vsg, slots.to(dev()))
    want = q[..., 7].double() * ref.values(kc, ks)[:, :, 7].view(n, 1, 1) / math.sqrt(D)
    # steps of the score: the scale, the product and two factors of ln 2, with their results; of 1: argument and result of
    # the exponential (two), the logarithm (two), and two sums
    assert ((lse.cpu().double() - want).abs() <= (6 * want.abs() + 8) * ref.U32).all()
