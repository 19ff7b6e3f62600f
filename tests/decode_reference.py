"""The operators around the selection in plain 64-bit form on the CPU, and the error bounds of their kernels.

Every function takes CPU tensors.  Bounds follow from the arithmetic: 32-bit sums, one rounding of the result, and the
roundings that each kernel's description names.
"""
import math

import torch

U32 = 2.0 ** -24  # half a step of a 32-bit float, relative

_CODES = torch.tensor([math.nan if (c & 127) == 127 else (-1.0 if c >> 7 else 1.0)
                       * ((c & 7) * 2.0 ** -9 if ((c >> 3) & 15) == 0 else (8 + (c & 7)) * 2.0 ** (((c >> 3) & 15) - 10))
                       for c in range(256)], dtype=torch.float64)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def values(codes, scales):
    """Cache rows in 64 bits."""
    v = _CODES[codes.view(torch.uint8).long()]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def quantise(x):
    """(codes uint8, scales uint8) of rows of finite values, nearest code by search, ties to the even code."""
    x = x.double().unflatten(-1, (-1, 32))
    top = x.abs().amax(-1)
    e = torch.full(top.shape, -126, dtype=torch.int64)
    for k in range(-126, 119):
        e = torch.where(top > 448 * 2.0 ** k, k + 1, e)
    e = torch.where(top == 0, -9, e)
    y = (x * torch.exp2(-e.double()).unsqueeze(-1)).clamp(-448, 448)
    size = _CODES[:127]
    hi = torch.searchsorted(size, y.abs().contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = size[hi] - y.abs(), y.abs() - size[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = torch.where(torch.signbit(y), code + 128, code)
    return code.flatten(-2).to(torch.uint8), (e + 127).to(torch.uint8)


def rope(x, positions, inv_freq, layout, offset, scale, inverse):
    """(result, bound of the error before the final rounding)."""
    y = x.double().clone()
    R = 2 * inv_freq.numel()
    size = torch.zeros_like(y)
    if R:
        angle = positions.double()[:, None] * inv_freq
        c, s = angle.cos()[:, None] * scale, angle.sin()[:, None] * scale * (-1 if inverse else 1)
        i = torch.arange(R // 2)
        ia, ib = (offset + 2 * i, offset + 2 * i + 1) if layout == "interleaved" else (offset + i, offset + R // 2 + i)
        a, b = x.double()[..., ia], x.double()[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * abs(scale)
    # angle rounded to 32 bits of half a turn (pi 2^-24), sine and cosine to two steps, times scale, products and sum
    return y, size * (math.pi + 4 + 1 + 2) * U32


def slots_of(table, page, positions):
    return table[positions // page].long() * page + positions % page


def gather(codes, scales, slots):
    """(values [n, H, D] in 64 bits, inside) of the slots; zeros outside."""
    inside = (slots >= 0) & (slots < codes.shape[0])
    at = torch.where(inside, slots, 0).long()
    v = torch.zeros(len(at), codes.shape[1], codes.shape[2], dtype=torch.float64)
    if inside.any():
        v[inside] = values(codes[at[inside]], scales[at[inside]])
    return v, inside


def index_scores(q, weights, codes, scales, table, lens, page, L):
    """(result [B * T, L], bound)."""
    B, T, H, D = q.shape
    out = torch.full((B, T, L), -math.inf, dtype=torch.float64)
    bound = torch.zeros(B, T, L, dtype=torch.float64)
    for b in range(B):
        n = max(0, min(int(lens[b]), L))
        if n == 0:
            continue
        k, inside = gather(codes, scales, slots_of(table[b], page, torch.arange(n)))
        k = k[:, 0]
        for t in range(T):
            qd, w = q[b, t].double(), weights[b, t].double()
            r = (k @ qd.t()).clamp(min=0) @ w
            out[b, t, :n] = torch.where(inside, r, -math.inf)
            # each step of the D- and H-long sums off by at most 2^-23 of the terms' sizes; fp16 queries: blocks far below
            # a row's largest lose bits beneath 2^-33 of it
            err = (k.abs() @ qd.abs().t()) * (D + H + 4) * 2 * U32
            err = err + k.abs().amax(1, keepdim=True) * qd.abs().sum(1) * 2.0 ** -33
            bound[b, t, :n] = err @ w.abs()
    return out.view(B * T, L), bound.view(B * T, L)


def attend(q, kc, ks, vc, vs, lists, tree_slots=None, tree_mask=None):
    """lists[b][t]: slots a token sees (before the tree's).  (out, lse, bound of out before its rounding, of lse)."""
    B, T, Hq, D = q.shape
    Hkv, Dv = kc.shape[1], vc.shape[2]
    G = Hq // Hkv
    out = torch.zeros(B, T, Hq, Dv, dtype=torch.float64)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64)
    eo, el = torch.zeros_like(out), torch.zeros_like(lse)
    p_step = half_step(torch.bfloat16) if q.dtype == torch.bfloat16 else half_step(torch.bfloat16) ** 2
    for b in range(B):
        for t in range(T):
            s = lists[b][t].long()
            if tree_slots is not None:
                line = [j for j in range(T) if (int(tree_mask[b, t]) >> j) & 1]
                s = torch.cat((s, tree_slots[b][line].long()))
            s = s[(s >= 0) & (s < kc.shape[0])]
            if not len(s):
                continue
            k, v = gather(kc, ks, s)[0], gather(vc, vs, s)[0]
            for h in range(Hq):
                kk, vv, qq = k[:, h // G], v[:, h // G], q[b, t, h].double()
                x = kk @ qq / math.sqrt(D)
                lse[b, t, h] = x.logsumexp(0)
                p = x.softmax(0)
                out[b, t, h] = p @ vv
                ex = (kk.abs() @ qq.abs()).max() / math.sqrt(D) * (D + 8) * 2 * U32
                ex = ex + (kk.abs().max() * qq.abs().sum() / math.sqrt(D)) * 2.0 ** -33
                # exponentials: argument rounded (its size in steps), result to two steps
                e_p = 2 * ex + 4 * U32 * (1 + x.abs().max())
                eo[b, t, h] = (p @ vv.abs()) * (p_step + 2 * e_p + (len(s) + 16) * 4 * U32)
                el[b, t, h] = e_p + (len(s) + 16) * 4 * U32 + 4 * U32 * x.logsumexp(0).abs()
    return out, lse, eo, el
