"""The operators of a speculative step in plain 64-bit form on the CPU: loops over sequences, blocks and nodes."""
import math

import torch

from tests import decode_reference as ref

LOW, HIGH = -126, 119


def spread(scales, S, D):
    """A block cache's scales as the 32-channel cache has them: [S, H, D / 32]."""
    block = S // scales.shape[0] if S else 1
    return scales.repeat_interleave(block, 0).unsqueeze(-1).expand(-1, -1, D // 32)


def encode(y):
    """Codes of values in units of the scale: nearest, ties to the even code; limited to +-448; no number stays none."""
    y = y.double()
    none = torch.isnan(y)
    y = torch.where(none, 0.0, y.clamp(-448, 448))
    size = ref._CODES[:127]
    hi = torch.searchsorted(size, y.abs().contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = size[hi] - y.abs(), y.abs() - size[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = torch.where(torch.signbit(y), code + 128, code)
    return torch.where(none, 127, code).to(torch.uint8)


def exponent(top):
    e = LOW
    while e < HIGH and top > 448 * 2.0 ** e:
        e += 1
    return e


def place(row, page, pages, at):
    """Slot of a position, or -1."""
    if at < 0 or at >= len(row) * page:
        return -1
    number = int(row[at // page])
    return number * page + at % page if 0 <= number < pages else -1


def store(x, codes, scales, row, first, count, page):
    """Rows x [count, H, D] in 64 bits to positions first ..: codes and scales (CPU, bytes) are changed."""
    S, H, D = codes.shape
    block, pages = S // scales.shape[0], S // page
    end = first + count
    start = first // block * block
    while start < end:
        slot = place(row, page, pages, start)
        if slot >= 0:
            low, high = max(first, start), min(end, start + block)
            for h in range(H):
                new = x[low - first:high - first, h]
                fine = new.abs()[torch.isfinite(new)]
                e = exponent(float(fine.max()) if fine.numel() else 0.0)
                if low > start:
                    before = int(scales[slot // block, h]) - 127
                    e = max(e, before)
                    if e > before:
                        old = ref._CODES[codes[slot:slot + low - start, h].long()]
                        codes[slot:slot + low - start, h] = encode(old * 2.0 ** (before - e))
                codes[slot + low - start:slot + high - start, h] = encode(new * 2.0 ** -e)
                scales[slot // block, h] = e + 127
        start += block


def block_write(x, codes, scales, table, first, counts, page):
    codes, scales = codes.clone(), scales.clone()
    for b in range(x.shape[0]):
        n = min(int(counts[b]), x.shape[1])
        if n > 0 and int(first[b]) >= 0:
            store(x[b, :n].double(), codes, scales, table[b], int(first[b]), n, page)
    return codes, scales


def block_keep(codes, scales, table, first, path, counts, page):
    codes, scales = codes.clone(), scales.clone()
    S, H, D = codes.shape
    for b in range(path.shape[0]):
        T = path.shape[1]
        n, at = min(int(counts[b]), T), int(first[b])
        if n <= 0 or at < 0:
            continue
        line = path[b, :n].tolist()
        same = 0
        while same < n and line[same] == same:
            same += 1
        rows = torch.zeros(n - same, H, D, dtype=torch.float64)
        for i in range(same, n):
            slot = place(table[b], page, S // page, at + line[i]) if 0 <= line[i] < T else -1
            if slot >= 0:
                scale = torch.exp2(scales[slot // (S // scales.shape[0])].double() - 127)
                rows[i - same] = ref._CODES[codes[slot].long()] * scale[:, None]
        store(rows, codes, scales, table[b], at + same, n - same, page)
    return codes, scales


def seen(table, page, pages, lens, L, T, first=None, mask=None):
    """lists[b][t] of slots that each token sees."""
    lists = []
    for b in range(len(lens)):
        n = max(0, min(int(lens[b]), L))
        slots = [place(table[b], page, pages, p) for p in range(n)]
        rows = []
        for t in range(T):
            if first is None:
                row = slots
            else:
                at = int(first[b])
                if at + t >= n:
                    row = []
                elif mask is None:
                    row = slots[:max(0, at + t + 1)]
                else:
                    bits = int(mask[b, t]) & ((1 << T) - 1)
                    row = slots[:max(0, at)] + [slots[at + j] for j in range(T) if bits >> j & 1 and 0 <= at + j < n]
            rows.append(torch.tensor(row, dtype=torch.int64))
        lists.append(rows)
    return lists


def attend(q, kc, ks, vc, vs, lists):
    """ref.attend with the bound of probabilities that are the sum of two bf16 numbers."""
    return ref.attend(q.float(), kc, spread(ks, kc.shape[0], kc.shape[2]), vc, spread(vs, vc.shape[0], vc.shape[2]), lists)


def clean(x):
    x = float(x)
    return x if 0 < x < math.inf else 0.0


def verify(probs, tokens, uniform, draft=None, mask=None, lens=None):
    """(tokens, path, counts) as lists of python numbers."""
    B, T, V = probs.shape
    out = []
    for b in range(B):
        n = T if lens is None else min(int(lens[b]), T)
        if n <= 0:
            out.append(([-1] * T, [-1] * T, 0))
            continue
        bits = [((1 << t) - 1 if mask is None else int(mask[b, t])) & ((1 << t) - 1) for t in range(T)]
        above = [(t - 1 if mask is None else line.bit_length() - 1) for t, line in enumerate(bits)]
        x, u = tokens[b].tolist(), [float(v) for v in uniform[b]]
        a, path = 0, [0]
        while True:
            kids = [t for t in range(1, n) if above[t] == a]
            rest, gone, found = 1.0, [], -1
            for c in kids:
                w = clean(probs[b, a, x[c]]) if 0 <= x[c] < V and x[c] not in gone else 0.0
                q = rest if draft is None else (clean(draft[b, c - 1, x[c]]) if 0 <= x[c] < V else 0.0)
                if u[c] * q < w:
                    found = c
                    break
                rest -= w
                gone.append(x[c])
            if found < 0:
                break
            a = found
            path.append(a)
        whole = [clean(v) for v in probs[b, a]]
        w = list(whole)
        if kids and draft is not None:
            w = [max(p - clean(d), 0.0) for p, d in zip(whole, draft[b, a])]
        elif kids:
            for c in kids:
                if 0 <= x[c] < V:
                    w[x[c]] = 0.0
        if sum(w) == 0:
            w = whole
        total = math.fsum(w)
        mark = total * min(max(u[0], 0.0), 1.0) if u[0] == u[0] else total
        run, new = 0.0, -1
        for v in range(V):
            if w[v] > 0:
                run += w[v]
                new = v
                if run > mark:
                    break
        line = [x[t] for t in path[1:]] + [new]
        out.append((line + [-1] * (T - len(line)), path + [-1] * (T - len(path)), len(path)))
    return tuple(torch.tensor([row[i] for row in out], dtype=torch.int32) for i in range(3))


def extend(refs, table, lens, page):
    refs, table, P = refs.tolist(), table.tolist(), len(refs)
    free, lacking = iter([i for i in range(P) if refs[i] <= 0]), []
    for row, n in zip(table, lens.tolist()):
        short = 0
        for j in range(min(-(-max(n, 0) // page), len(row))):
            if not 0 <= row[j] < P:
                row[j] = next(free, -1)
                if row[j] < 0:
                    short += 1
                else:
                    refs[row[j]] = 1
        lacking.append(short)
    return refs, table, lacking


def release(refs, table, lens, page):
    refs, table, P = refs.tolist(), table.tolist(), len(refs)
    for row, n in zip(table, lens.tolist()):
        for j in range(min(-(-max(n, 0) // page), len(row)), len(row)):
            if 0 <= row[j] < P:
                refs[row[j]] -= 1
            row[j] = -1
    return refs, table


def fork(refs, table, lens, page, parents, M):
    """(refs, rows, lacking, pairs of pages (from, to))."""
    refs, table, lens, P = refs.tolist(), table.tolist(), lens.tolist(), len(refs)
    free, rows, lacking, pairs = iter([i for i in range(P) if refs[i] <= 0]), [], [], []
    for b in parents.tolist():
        row, short = [-1] * M, 0
        if 0 <= b < len(table):
            n = max(lens[b], 0)
            full = n // page
            for j in range(min(full, M, len(table[b]))):
                if 0 <= table[b][j] < P:
                    row[j] = table[b][j]
                    refs[row[j]] += 1
            if n % page and full < M and full < len(table[b]) and 0 <= table[b][full] < P:
                row[full] = next(free, -1)
                short = int(row[full] < 0)
                if not short:
                    refs[row[full]] = 1
                    pairs.append((table[b][full], row[full]))
        rows.append(row)
        lacking.append(short)
    return refs, rows, lacking, pairs


def compact(refs, table):
    refs, table, P = refs.tolist(), table.tolist(), len(refs)
    used = sum(r > 0 for r in refs)
    pairs = list(zip([i for i in range(used, P) if refs[i] > 0], [i for i in range(used) if refs[i] <= 0]))
    to = dict(pairs)
    moved = [to.get(i, i) if refs[i] > 0 else -1 for i in range(P)]
    table = [[moved[e] if 0 <= e < P else e for e in row] for row in table]
    for a, b in pairs:
        refs[b], refs[a] = refs[a], 0
    return refs, table, moved, pairs
