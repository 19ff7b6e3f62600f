"""The operators of a speculative decode step over a pool of cache pages, case by case: attention over a cache with one
scale for a block of tokens and a head, the writes that make and tidy that cache, the verification of drafted tokens, and
the pool's pages: taking, forking and compacting them.

A block cache is e4m3 codes [S, H, D] with one power-of-two scale byte s for each N slots and head, [S / N, H]:
value = code * 2^(s - 127).
"""
import math

import torch

own = False

LOW, HIGH = -126, 119  # exponents a block's scale may have
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one sequence's next token over a short cache: latency
        dict(name="attend_token", op="attend", B=1, T=1, Hq=32, Hkv=8, D=128, Dv=128, L=2047, page=16, block=16, form="all",
             dtype="bf16"),
        # the next token of 64 sequences
        dict(name="attend_batch", op="attend", B=64, T=1, Hq=32, Hkv=8, D=128, Dv=128, L=8192, page=64, block=64, form="all",
             dtype="bf16"),
        # trees of 13 drafted tokens behind long prefixes, an odd head width, pages that end inside a tile
        dict(name="attend_tree", op="attend", B=12, T=13, Hq=32, Hkv=4, D=96, Dv=96, L=10007, page=48, block=16, form="tree",
             dtype="fp16"),
        # pieces of two prompts over what is cached of them
        dict(name="attend_prompt", op="attend", B=2, T=1000, Hq=32, Hkv=8, D=128, Dv=128, L=8192, page=64, block=64,
             form="causal", dtype="bf16"),
        # one decode step of 64 sequences writes its keys
        dict(name="write_step", op="write", B=64, T=1, H=8, D=128, cap=8192, page=64, block=64, dtype="bf16"),
        # pieces of four prompts, cut at odd places
        dict(name="write_prompt", op="write", B=4, T=8192, H=8, D=128, cap=16384, page=64, block=32, dtype="fp16"),
        # the accepted lines of 64 trees move up to where their sequences end
        dict(name="keep_step", op="keep", B=64, T=40, H=8, D=128, cap=4096, page=64, block=16),
        # five drafted tokens of 64 sequences against their draft model's probabilities
        dict(name="verify_chain", op="verify", B=64, T=6, V=128000, tree=False, draft=True, dtype="fp32"),
        # trees of 31 tokens that are no samples, a half-precision target
        dict(name="verify_tree", op="verify", B=8, T=32, V=50001, tree=True, draft=False, dtype="bf16"),
        # rows of a batch that grow by their next pages
        dict(name="pages_extend", op="pages", kind="extend", B=256, M=256, P=32768, page=64, H=0, D=0, block=64, n=0),
        # each of 32 prompts branches into four answers
        dict(name="pages_fork", op="pages", kind="fork", B=32, M=128, P=6144, page=64, H=8, D=128, block=64, n=128),
        # a pool that is half free is drawn together
        dict(name="pages_compact", op="pages", kind="compact", B=64, M=96, P=8192, page=64, H=8, D=128, block=64, n=0),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, evenly over the logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    while True:  # a case that costs no more than the largest listed ones
        case = _drawn(rng)
        cost = work(case)
        if cost["bytes"] <= 6e8 and cost["flops"] <= 1e11:
            return case


def _drawn(rng):
    op = rng.choice(("attend", "attend", "attend", "write", "write", "keep", "verify", "verify", "pages", "pages"))
    block = rng.choice((1, 8, 16, 16, 32, 64, 64, 100))
    page = block * rng.choice((1, 1, 2, 3, 4))
    H, D = rng.choice((1, 2, 4, 5, 8)), 32 * rng.choice((1, 2, 3, 4, 4, 5, 8))
    if op == "attend":
        form = rng.choice(("all", "tree", "causal"))
        B = _spread(rng, 1, 64)
        T = rng.choice((1, 1, 2, 5)) if form == "all" else _spread(rng, 2, 64) if form == "tree" else _spread(rng, 1, 2048)
        L = _spread(rng, T, max(T, min(131072, (1 << 30) // (B * H * D))))
        return dict(op=op, B=B, T=T, Hq=H * _spread(rng, 1, 64 // H), Hkv=H, D=D, Dv=rng.choice((D, D, 32 * rng.randint(1, 8))),
                    L=L, page=page, block=block, form=form, dtype=rng.choice(("bf16", "fp16")))
    if op == "write":
        B, T = _spread(rng, 1, 64), _spread(rng, 1, 8192)
        return dict(op=op, B=B, T=T, H=H, D=D, cap=T + _spread(rng, 1, 4096), page=page, block=block,
                    dtype=rng.choice(tuple(TYPES)))
    if op == "keep":
        block = min(block, 32)
        page, T = block * rng.choice((1, 1, 2, 3, 4)), rng.randint(block + 4, 64)
        return dict(op=op, B=_spread(rng, 1, 256), T=T, H=H, D=D, cap=T + _spread(rng, 1, 4096), page=page, block=block)
    if op == "verify":
        tree, draft = rng.choice(((False, True), (False, True), (False, False), (True, False)))
        B, T, V = _spread(rng, 1, 128), _spread(rng, 1, 64), _spread(rng, 16, 200000)
        return dict(op=op, B=B, T=min(T, max(1, (1 << 27) // (B * V))), V=V, tree=tree, draft=draft, dtype=rng.choice(tuple(TYPES)))
    kind = rng.choice(("extend", "free", "fork", "compact", "copy"))
    B, M = _spread(rng, 1, 256), _spread(rng, 1, 256)
    if kind in ("extend", "free"):
        return dict(op=op, kind=kind, B=B, M=M, P=B * M + _spread(rng, 1, 32768), page=page, H=0, D=0, block=block, n=0)
    P = _spread(rng, 4, max(4, min(8192, (1 << 29) // (page * H * D))))
    M = min(M, max(1, P // B))
    return dict(op=op, kind=kind, B=min(B, P), M=M, P=P, page=page, H=H, D=D, block=block,
                n=0 if kind == "compact" else _spread(rng, 1, max(1, P // 4)))


# ---- inputs

def _exponent(top):
    """The smallest e with top <= 448 * 2^e; the lowest one for a block of zeros."""
    m, p = torch.frexp(top)
    e = torch.where(m <= 0.875, p - 9, p - 8)
    return torch.where(top > 0, e, LOW).clamp(LOW, HIGH)


def _cache(S, H, D, block, g):
    """A filled cache (codes, scale bytes): normal values, a few channels several times larger than the rest, rows of differing size."""
    channel = 1 + 7 * (torch.rand(D, generator=g, device="cuda") > 0.97)
    codes = torch.empty((S, H, D), dtype=torch.uint8, device="cuda")
    scales = torch.empty((S // block, H), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (block * H * D))
    for at in range(0, S // block, step):  # a piece at a time: temporaries are several times the cache
        n = min(step, S // block - at)
        x = torch.randn(n, block, H, D, generator=g, device="cuda") * channel
        x *= torch.exp(0.5 * torch.randn(n, block, 1, 1, generator=g, device="cuda"))
        e = _exponent(x.abs().amax((1, 3)))
        code = torch.ldexp(x, -e[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        codes[at * block:(at + n) * block] = code.view(torch.uint8).flatten(0, 1)
        scales[at:at + n] = (e + 127).to(torch.uint8)
    return codes.view(torch.float8_e4m3fn), scales


def _pages(B, L, page, g):
    """(page table of B sequences with room for L positions each, slots of the cache): pages in random order."""
    per = -(-L // page)
    return torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per), B * per * page


def _between(low, high, n, g):
    """int32 [n] evenly between low and high, both among them."""
    return torch.randint(low, high + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _kept(c):
    """(most rows that a line keeps, first row of those that move up)"""
    most = (c["T"] - c["block"] + 1) // 2
    return most, most + c["block"] - 1


def _tree(B, T, g):
    """Ancestor bits int64 [B, T]: each token hangs on an earlier one, and sees itself and its line."""
    mask = torch.ones(B, T, dtype=torch.int64, device="cuda")
    for t in range(1, T):
        parent = torch.randint(0, t, (B, 1), generator=g, device="cuda")
        mask[:, t] = mask.gather(1, parent)[:, 0] | (1 << t if t < 63 else -(1 << 63))
    return mask


def _probabilities(shape, dtype, g):
    """A model's distributions: few likely tokens, many unlikely ones."""
    return torch.softmax(3 * torch.randn(shape, generator=g, device="cuda"), -1).to(TYPES[dtype])


def _table(c, share, g):
    """(refs, table) of a pool of which a share is in use: rows of differing length, pages in random order, some of them
    held by two rows."""
    B, M, P = c["B"], c["M"], c["P"]
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    count = (torch.rand(B, generator=g, device="cuda") * (2 * share) * min(M, P // B)).clamp(max=min(M, P // B)).int()
    order = torch.randperm(P, generator=g, device="cuda")[:B * min(M, P // B)].view(B, -1)
    if order.shape[1] < M:
        order = torch.cat((order, order.new_zeros(B, M - order.shape[1])), 1)
    at = torch.arange(M, device="cuda")
    if B > 1:
        order[1] = torch.where(at < torch.minimum(count[0], count[1]) // 2, order[0], order[1])
    table = torch.where(at < count[:, None], order, -1).to(torch.int32)
    refs += torch.bincount(table[table >= 0].long(), minlength=P).int()
    return refs, table


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, s = case, {"case": case}
    if c["op"] == "attend":
        B, T, L = c["B"], c["T"], c["L"]
        s["q"] = torch.randn((B, T, c["Hq"], c["D"]), generator=g, device="cuda").to(TYPES[c["dtype"]])
        s["page_table"], S = _pages(B, L, c["page"], g)
        s["k_codes"], s["k_scales"] = _cache(S, c["Hkv"], c["D"], c["block"], g)
        s["v_codes"], s["v_scales"] = _cache(S, c["Hkv"], c["Dv"], c["block"], g)
        s["seq_lens"] = _between((L + 1) // 2, L, B, g)
        s["seq_lens"][0] = L
        s["first"] = s["tree_mask"] = None
        if c["form"] != "all":  # the tokens' own rows are the last ones; a short sequence's last tokens are padding
            s["seq_lens"] = s["seq_lens"].clamp(min=T)
            s["first"] = s["seq_lens"] - T
            if B > 1:
                s["first"][1] += T // 3
        if c["form"] == "tree":
            s["tree_mask"] = _tree(B, T, g)
    elif c["op"] in ("write", "keep"):
        B, T = c["B"], c["T"]
        s["page_table"], S = _pages(B, c["cap"], c["page"], g)
        s["codes"], s["scales"] = _cache(S, c["H"], c["D"], c["block"], g)
        s["first"] = _between(0, c["cap"] - T, B, g)
        if c["op"] == "write":
            size = torch.exp(1.5 * torch.randn(B, 1, 1, 1, generator=g, device="cuda"))  # some outgrow their block's scale
            s["x"] = (torch.randn((B, T, c["H"], c["D"]), generator=g, device="cuda") * size).to(TYPES[c["dtype"]])
            s["counts"] = _between((T + 1) // 2, T, B, g)
            if B > 8:
                s["counts"][5] = 0
        else:
            # lines of broad trees: the root, perhaps a first child, then rows from blocks behind all that is kept (so that
            # a pass can be repeated)
            most, behind = _kept(c)
            s["counts"] = _between(1, most, B, g)
            later = torch.rand(B, T - behind, generator=g, device="cuda").argsort(1)[:, :most].sort(1).values + behind
            start = _between(1, 2, B, g)[:, None]
            at = torch.arange(most, device="cuda")
            line = torch.where(at < start, at, later)
            s["path"] = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
            s["path"][:, :most] = torch.where(at < s["counts"][:, None], line, -1).to(torch.int32)
    elif c["op"] == "verify":
        B, T, V = c["B"], c["T"], c["V"]
        s["probs"] = _probabilities((B, T, V), c["dtype"], g)
        s["uniform"] = torch.rand((B, T), generator=g, device="cuda")
        s["tree_mask"] = _tree(B, T, g) if c["tree"] else None
        s["draft_probs"] = None
        if c["draft"]:  # a draft that resembles the target, and its samples
            near = s["probs"][:, :T - 1].float() * torch.exp(0.7 * torch.randn((B, T - 1, V), generator=g, device="cuda"))
            s["draft_probs"] = (near / near.sum(-1, keepdim=True)).to(TYPES[c["dtype"]])
            source = s["draft_probs"].float()
        else:  # likely tokens
            parent = _parents(s["tree_mask"], B, T)[:, 1:].long()
            source = s["probs"].gather(1, parent[..., None].expand(-1, -1, V)).float() ** 2
        noise = -torch.log(torch.rand(source.shape, generator=g, device="cuda").clamp(min=1e-20))
        s["tokens"] = torch.zeros((B, T), dtype=torch.int32, device="cuda")
        if T > 1:
            s["tokens"][:, 1:] = (source / noise).argmax(-1)
        s["tokens"][:, 0] = _between(0, V - 1, B, g)
        s["lens"] = _between((T + 1) // 2, T, B, g)
    else:
        B, M, P, page = c["B"], c["M"], c["P"], c["page"]
        s["refs"], s["table"] = _table(c, {"extend": 0.3, "free": 0.5, "fork": 0.3, "compact": 0.5, "copy": 0.5}[c["kind"]], g)
        held = (s["table"] >= 0).sum(1)
        s["lens"] = None
        if c["kind"] == "extend":  # most rows grow by a page or two, some not at all
            s["lens"] = ((held + torch.randint(0, 3, (B,), generator=g, device="cuda")).clamp(max=M) * page).to(torch.int32)
        if c["kind"] == "free":  # a quarter of the sequences end, others drop pages behind their drafts
            keep = (held - torch.randint(0, 2, (B,), generator=g, device="cuda")).clamp(min=0)
            s["lens"] = (torch.where(torch.rand(B, generator=g, device="cuda") < 0.25, 0, keep) * page).to(torch.int32)
        if c["kind"] == "fork":
            s["lens"] = (held * page - torch.randint(0, page, (B,), generator=g, device="cuda")).clamp(min=0).to(torch.int32)
            s["parents"] = (torch.arange(c["n"], device="cuda") % B).to(torch.int32)
        if c["kind"] == "copy":
            both = torch.randperm(P, generator=g, device="cuda").to(torch.int32)[:2 * c["n"]]
            s["src"], s["dst"] = both[:both.numel() // 2].contiguous(), both[both.numel() // 2:][:both.numel() // 2].contiguous()
        if c["H"]:
            s["buffers"] = [torch.randint(0, 256, (P * page, c["H"], c["D"]), generator=g, device="cuda", dtype=torch.uint8)
                            for _ in "kv"]
            s["buffers"] += [torch.randint(1, 247, (P * page // c["block"], c["H"]), generator=g, device="cuda",
                                           dtype=torch.uint8) for _ in "kv"]
    return s


# ---- one pass

def _slots(table, page, positions):
    """Cache slots of positions [B, n] through the page table; -1 past its end."""
    inside = (positions >= 0) & (positions < table.shape[1] * page)
    at = torch.where(inside, positions, 0).long()
    slots = table.gather(1, at // page).long() * page + at % page
    return torch.where(inside, slots, -1)


def _values(codes, scales, slots):
    """Cache rows [B, n, H, D] in 32 bits."""
    e = scales[slots // (codes.shape[0] // scales.shape[0])].int() - 127
    return torch.ldexp(codes.view(torch.uint8)[slots].view(torch.float8_e4m3fn).float(), e.unsqueeze(-1))


def _seen(c, s):
    """[B, T, L]: which positions a token sees."""
    at = torch.arange(c["L"], device="cuda")
    seen = (at < s["seq_lens"].view(-1, 1, 1)).expand(c["B"], c["T"], -1)
    if s["first"] is None:
        return seen
    t = torch.arange(c["T"], device="cuda")
    behind = at - s["first"].view(-1, 1, 1)
    if s["tree_mask"] is None:
        mine = behind <= t.view(1, -1, 1)
    else:
        bit = (s["tree_mask"].unsqueeze(-1) >> behind.clamp(0, 63)) & 1
        mine = (behind < 0) | ((behind < c["T"]) & (bit == 1))
    alive = s["first"].view(-1, 1) + t < s["seq_lens"].view(-1, 1)
    return seen & mine & alive.unsqueeze(-1)


def _attend(s):
    c = s["case"]
    B, T, G = c["B"], c["T"], c["Hq"] // c["Hkv"]
    slots = _slots(s["page_table"], c["page"], torch.arange(c["L"], device="cuda").expand(B, -1))
    k = _values(s["k_codes"], s["k_scales"], slots).permute(0, 2, 3, 1).contiguous()   # [B, Hkv, D, L]
    v = _values(s["v_codes"], s["v_scales"], slots).transpose(1, 2).contiguous()       # [B, Hkv, L, Dv]
    q = s["q"].float().unflatten(2, (c["Hkv"], G)).transpose(1, 2).flatten(2, 3).contiguous()  # [B, Hkv, T * G, D]
    seen = _seen(c, s)[:, None, :, None].expand(B, 1, T, G, -1).flatten(2, 3)
    x = (torch.matmul(q, k) * c["D"] ** -0.5).masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    lse = torch.where(total == 0, -math.inf, top + total.log())
    out, lse = (y.unflatten(2, (T, G)).transpose(1, 2) for y in (out, lse))
    return {"out": out.reshape(B, T, c["Hq"], -1).to(s["q"].dtype), "lse": lse.reshape(B, T, c["Hq"])}


def _store(x, counts, s):
    """Rows x [B, T, H, D] in 32 bits to positions first .. of their sequences."""
    c, codes, scales = s["case"], s["codes"].view(torch.uint8), s["scales"]
    block, first = c["block"], s["first"].view(-1, 1)
    t = torch.arange(x.shape[1], device="cuda")
    slots = _slots(s["page_table"], c["page"], first + t)
    valid = (t < counts.view(-1, 1)) & (slots >= 0)
    of = torch.where(valid, slots // block, 0)
    top = x.abs().amax(-1) * valid.unsqueeze(-1)
    tops = torch.zeros(scales.shape, device="cuda").scatter_reduce_(
        0, of.flatten().unsqueeze(-1).expand(-1, c["H"]), top.flatten(0, 1), "amax")
    # rows that stay before the first new one
    start = torch.where(valid[:, 0], slots[:, 0] // block, 0)
    stay = (torch.arange(block, device="cuda") < first % block) & valid[:, :1]
    e = _exponent(tops)
    floor = torch.where(stay[:, :1], scales[start].int() - 127, LOW)
    e.scatter_reduce_(0, start.unsqueeze(-1).expand(-1, c["H"]), floor.int(), "amax")
    rows = start.unsqueeze(-1) * block + torch.arange(block, device="cuda")
    old = codes[rows].view(torch.float8_e4m3fn).float()
    shift = scales[start].int() - 127 - e[start]
    again = torch.ldexp(old, shift[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    new = torch.ldexp(x, -e[of].unsqueeze(-1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[rows[stay]] = again[stay]
    codes[slots[valid]] = new[valid]
    scales[of[valid]] = (e + 127).to(torch.uint8)[of[valid]]


def _keep(s):
    """As rows from the first that moves on."""
    c = s["case"]
    t = torch.arange(c["T"], device="cuda")
    path = torch.where(t < s["counts"].view(-1, 1), s["path"], t)
    slots = _slots(s["page_table"], c["page"], s["first"].view(-1, 1) + path)
    x = _values(s["codes"], s["scales"], slots)
    same = (path == t).cumprod(1).sum(1, dtype=torch.int32)  # rows that stay where they are
    at = (same.view(-1, 1) + t).clamp(max=c["T"] - 1).long()
    x = x.gather(1, at[..., None, None].expand_as(x))
    moved = dict(s, first=s["first"] + same)
    _store(x, s["counts"] - same, moved)


def _parents(tree_mask, B, T):
    """int64 [B, T]: the highest earlier node of each line; -1 where there is none."""
    t = torch.arange(T, device="cuda")
    if tree_mask is None:
        return (t - 1).expand(B, -1)
    bits = ((tree_mask.unsqueeze(-1) >> t) & 1) * (t + 1) * (t < t.view(-1, 1))
    return bits.amax(-1) - 1


def _verify(s):
    c = s["case"]
    B, T, V = c["B"], c["T"], c["V"]
    b = torch.arange(B, device="cuda")
    x, u, parent = s["tokens"].long(), s["uniform"].double(), _parents(s["tree_mask"], B, T)
    p = s["probs"][b[:, None], parent.clamp(min=0), x].double()  # of each node's token, after its parent
    q = None if s["draft_probs"] is None else s["draft_probs"][b[:, None], torch.arange(T - 1, device="cuda"), x[:, 1:]].double()
    same = (x[:, :, None] == x[:, None]) & (parent[:, :, None] == parent[:, None])
    again = (same & torch.ones(T, T, dtype=torch.bool, device="cuda").tril(-1)).any(-1)
    p = torch.where(again, 0.0, p)
    node = torch.zeros(B, dtype=torch.int64, device="cuda")
    count = torch.ones(B, dtype=torch.int64, device="cuda")
    rest = torch.ones(B, dtype=torch.float64, device="cuda")
    path = torch.full((B, T), -1, dtype=torch.int64, device="cuda")
    path[:, 0] = 0
    for t in range(1, T):
        child = (parent[:, t] == node) & (t < s["lens"])
        if q is None:
            taken = child & (u[:, t] * rest < p[:, t])
            rest = torch.where(taken, 1.0, torch.where(child, rest - p[:, t], rest))
        else:
            taken = child & (u[:, t] * q[:, t - 1] < p[:, t])
        at = count.clamp(max=T - 1)
        path[b, at] = torch.where(taken, t, path[b, at])
        count = count + taken
        node = torch.where(taken, t, node)
    w = s["probs"][b, node].double()
    whole = w
    if q is None:
        off = (parent == node[:, None]) & (torch.arange(T, device="cuda") < s["lens"][:, None])
        w = w.masked_fill(torch.zeros_like(w).scatter_reduce_(1, x, off.double(), "amax") > 0, 0.0)
    else:
        refused = node + 1 < s["lens"]
        if T > 1:
            less = (w - s["draft_probs"][b, node.clamp(max=T - 2)].double()).clamp(min=0)
            w = torch.where(refused[:, None], less, w)
    w = torch.where((w.sum(-1) == 0)[:, None], whole, w)
    run = w.cumsum(-1)
    new = (run <= u[:, :1] * run[:, -1:]).sum(-1).clamp(max=V - 1)
    out = torch.where(path[:, 1:] >= 0, x.gather(1, path[:, 1:].clamp(min=0)), -1)
    out = torch.cat((out, out.new_full((B, 1), -1)), 1)
    out[b, count - 1] = new
    return {"tokens": out.int(), "path": path.int(), "counts": count.int()}


def _page_view(buffer, P):
    return buffer.view(P, -1)


def _take(refs, table, lens, page):
    """Missing entries for `lens` positions, in order, get the lowest free pages; pages that each row lacks."""
    at = torch.arange(table.shape[1], device="cuda")
    missing = (table < 0) & (at < ((lens + page - 1) // page).view(-1, 1))
    rank = missing.flatten().cumsum(0).view_as(table) - 1
    pages = torch.arange(refs.numel(), device="cuda")
    free = torch.where(refs <= 0, pages, refs.numel()).sort().values
    got = free[rank.clamp(0, refs.numel() - 1)]
    there = missing & (rank < refs.numel()) & (got < refs.numel())
    table.copy_(torch.where(there, got, table))
    refs.scatter_add_(0, torch.where(there, got, 0).flatten(), there.flatten().int())
    return (missing & ~there).sum(1).int()


def _on_pages(s):
    c = s["case"]
    kind, page, P = c["kind"], c["page"], c["P"]
    if kind == "copy":
        for buffer in s["buffers"]:
            rows = _page_view(buffer, P)
            rows[s["dst"].long()] = rows[s["src"].long()]
        return s["buffers"]
    refs, table = s["refs"].clone(), s["table"].clone()
    at = torch.arange(c["M"], device="cuda")
    if kind == "extend":
        return {"refs": refs, "table": table, "lacking": _take(refs, table, s["lens"], page)}
    if kind == "free":
        go = (at >= ((s["lens"] + page - 1) // page).view(-1, 1)) & (table >= 0)
        refs.scatter_add_(0, torch.where(go, table, 0).flatten().long(), -go.flatten().int())
        table.masked_fill_(go, -1)
        return {"refs": refs, "table": table}
    if kind == "fork":
        lens = s["lens"][s["parents"].long()].view(-1, 1)
        rows = table[s["parents"].long()]
        shared = (at < lens // page) & (rows >= 0)
        child = torch.where(shared, rows, -1)
        refs.scatter_add_(0, torch.where(shared, rows, 0).flatten().long(), shared.flatten().int())
        part = (lens % page != 0)[:, 0]
        last = (lens[:, 0] // page).clamp(max=c["M"] - 1).long()
        # only the last, partly filled page of a row is missing
        src = rows.gather(1, last.view(-1, 1))[:, 0].long()
        wanted = torch.where(part & (src >= 0), 1, 0).int()
        fresh = torch.full((rows.shape[0], 1), -1, dtype=torch.int32, device="cuda")
        lacking = _take(refs, fresh, wanted, 1)
        child.scatter_(1, last.view(-1, 1), torch.where(wanted.view(-1, 1) > 0, fresh, child.gather(1, last.view(-1, 1))))
        there = fresh[:, 0] >= 0
        for buffer in s["buffers"]:
            rows = _page_view(buffer, P)
            rows[fresh[there, 0].long()] = rows[src[there]]
        return {"refs": refs, "child": child, "lacking": lacking, "buffers": s["buffers"]}
    pages = torch.arange(P, device="cuda")
    used = refs > 0
    n = used.sum()
    src = torch.where(used & (pages >= n), pages, P).sort().values
    dst = torch.where(~used & (pages < n), pages, P).sort().values
    there = src < P
    src, dst = src[there], dst[there]
    for buffer in s["buffers"]:
        rows = _page_view(buffer, P)
        rows[dst] = rows[src]
    moved = torch.where(used, pages, -1)
    moved[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    table = torch.where(table >= 0, moved[table.clamp(min=0).long()], table).int()
    return {"refs": refs, "table": table, "moved": moved.int(), "buffers": s["buffers"]}


def _own(s):
    import exact_top_selection_amd as ets
    c = s["case"]
    if c["op"] == "attend":
        out, lse = ets.attend_blocks(s["q"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], s["page_table"],
                                     s["seq_lens"], c["page"], c["L"], first=s["first"], tree_mask=s["tree_mask"])
        return {"out": out, "lse": lse}
    if c["op"] == "write":
        ets.block_write(s["x"], s["codes"], s["scales"], s["page_table"], s["first"], s["counts"], c["page"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if c["op"] == "keep":
        ets.block_keep(s["codes"], s["scales"], s["page_table"], s["first"], s["path"], s["counts"], c["page"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if c["op"] == "verify":
        tokens, path, counts = ets.verify_drafts(s["probs"], s["tokens"], s["uniform"], draft_probs=s["draft_probs"],
                                                 tree_mask=s["tree_mask"], lens=s["lens"])
        return {"tokens": tokens, "path": path, "counts": counts}
    kind, page, P = c["kind"], c["page"], c["P"]
    if kind == "copy":
        ets.pages_copy(s["buffers"], s["src"], s["dst"], P)
        return s["buffers"]
    refs, table = s["refs"].clone(), s["table"].clone()  # the pass can be repeated; a program changes its own
    if kind == "extend":
        return {"refs": refs, "table": table, "lacking": ets.pages_extend(refs, table, s["lens"], page)}
    if kind == "free":
        ets.pages_free(refs, table, s["lens"], page)
        return {"refs": refs, "table": table}
    if kind == "fork":
        child, lacking = ets.pages_fork(refs, table, s["lens"], page, s["parents"], s["buffers"])
        return {"refs": refs, "child": child, "lacking": lacking, "buffers": s["buffers"]}
    moved = ets.pages_compact(refs, table, s["buffers"])
    return {"refs": refs, "table": table, "moved": moved, "buffers": s["buffers"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op in ("write", "keep"):
        if op == "write":
            _store(state["x"].float(), state["counts"], state)
        else:
            _keep(state)
        return {"codes": state["codes"], "scales": state["scales"]}
    return {"attend": _attend, "verify": _verify, "pages": _on_pages}[op](state)


# ---- what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "attend":
        B, T, L = c["B"], c["T"], c["L"]
        n = max((0.75 + 0.25 / B) * L, T if c["form"] != "all" else 0)  # lengths lie between L/2 and L, the first is L
        pairs = T * n - (0 if c["form"] == "all" else T * (T - 1) / 2 if c["form"] == "causal" else T * T / 2)
        return {"bytes": B * c["Hkv"] * n * (c["D"] + c["Dv"] + 2 / c["block"]) + 4 * B * n / c["page"]
                + B * T * c["Hq"] * (2 * (c["D"] + c["Dv"]) + 4), "flops": 2 * B * c["Hq"] * max(pairs, 1) * (c["D"] + c["Dv"])}
    if c["op"] == "write":
        n = 0.75 * c["B"] * c["T"] * c["H"]
        return {"bytes": n * (c["D"] * (SIZE[c["dtype"]] + 1) + 1 / c["block"]) + 8 * c["B"], "flops": 2 * n * c["D"]}
    if c["op"] == "keep":
        n = c["B"] * max(1, _kept(c)[0] / 2 - 1) * c["H"] * c["D"]  # rows that move
        return {"bytes": 2 * n + 4 * c["B"] * (c["T"] + 2), "flops": n}
    if c["op"] == "verify":
        rows = 2 if c["draft"] else 1
        return {"bytes": c["B"] * (rows * c["V"] * SIZE[c["dtype"]] + c["T"] * 20), "flops": c["B"] * c["V"] * rows}
    entries = 4 * (c["P"] + 2 * c["B"] * c["M"])
    held = c["page"] * c["H"] * c["D"] * 2 + 2 * (c["page"] // c["block"]) * c["H"]
    moved = {"copy": min(c["n"], c["P"] // 2), "fork": min(c["n"], c["P"] // 2), "compact": c["P"] // 4}.get(c["kind"], 0)
    return {"bytes": entries + 2 * moved * held, "flops": c["P"] + c["B"] * c["M"]}


# ---- the definitions in 64 bits

_E4M3 = None


def _decoded(codes, scales, block, slots):
    """Cache rows in 64 bits from the bits of their codes: sign, 4 bits of exponent, 3 of fraction."""
    global _E4M3
    if _E4M3 is None:
        table = []
        for byte in range(256):
            exponent, fraction = (byte >> 3) & 15, byte & 7
            size = fraction * 2.0 ** -9 if exponent == 0 else (8 + fraction) * 2.0 ** (exponent - 10)
            table.append(math.nan if byte & 127 == 127 else -size if byte >> 7 else size)
        _E4M3 = torch.tensor(table, dtype=torch.float64, device="cuda")
    value = _E4M3[codes.view(torch.uint8).index_select(0, slots).int()]
    return value * torch.exp2(scales.index_select(0, slots // block).double() - 127).unsqueeze(-1)


def _places(table_row, page, positions):
    return table_row[positions // page].long() * page + positions % page


def _exact_attend(c, s):
    out = torch.zeros(c["B"], c["T"], c["Hq"], c["Dv"], dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["T"], c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    G, root = c["Hq"] // c["Hkv"], math.sqrt(c["D"])
    for b, n in enumerate(s["seq_lens"].tolist()):
        slots = _places(s["page_table"][b], c["page"], torch.arange(n, device="cuda"))
        k = _decoded(s["k_codes"], s["k_scales"], c["block"], slots)
        v = _decoded(s["v_codes"], s["v_scales"], c["block"], slots)
        see = torch.ones(c["T"], n, dtype=torch.bool, device="cuda")
        if s["first"] is not None:
            start = int(s["first"][b])
            lines = [0] * c["T"] if s["tree_mask"] is None else s["tree_mask"][b].tolist()
            for t, line in enumerate(lines):
                if start + t >= n:
                    see[t] = False
                elif s["tree_mask"] is None:
                    see[t, start + t + 1:] = False
                else:
                    see[t, start:] = torch.tensor([j < c["T"] and bool(line >> j & 1) for j in range(n - start)], device="cuda")
        for h in range(c["Hq"]):
            kk, vv = k[:, h // G].contiguous(), v[:, h // G].contiguous()
            for t in range(0, c["T"], 256):
                x = s["q"][b, t:t + 256, h].double() @ kk.t().contiguous() / root
                x = x.masked_fill(~see[t:t + 256], -math.inf)
                lse[b, t:t + 256, h] = x.logsumexp(-1)
                out[b, t:t + 256, h] = torch.nan_to_num(x.softmax(-1)) @ vv
    return {"out": out, "lse": lse}


def _exact_store(c, s):
    """The value that each code rounds, in units of its block's scale."""
    block = c["block"]
    codes, scales = s["codes"].double(), s["scales"].clone()
    for b, (first, count) in enumerate(zip(s["first"].tolist(), s["counts"].tolist())):
        if c["op"] == "keep":
            line = s["path"][b, :count].tolist()
            same = 0
            while same < count and line[same] == same:
                same += 1
            source = _places(s["page_table"][b], c["page"], torch.tensor([first + j for j in line[same:]], dtype=torch.int64, device="cuda"))
            x = _decoded(s["codes"], s["scales"], block, source)
            first, count = first + same, count - same
        else:
            x = s["x"][b, :count].double()
        if count <= 0:
            continue
        slots = _places(s["page_table"][b], c["page"], torch.arange(first, first + count, device="cuda"))
        stay = first % block
        of = torch.unique_consecutive(slots // block)
        sizes = torch.zeros(len(of), c["H"], dtype=torch.float64, device="cuda")
        index = (torch.arange(count, device="cuda") + stay) // block
        sizes.scatter_reduce_(0, index[:, None].expand(-1, c["H"]), x.abs().amax(-1), "amax")
        e = torch.where(sizes > 0, torch.ceil(torch.log2(sizes / 448)), float(LOW)).clamp(LOW, HIGH)
        if stay:
            before = scales[of[0]].double() - 127
            e[0] = torch.maximum(e[0], before)
            old = torch.arange(stay, device="cuda") + of[0] * block
            codes[old] = codes[old] * torch.exp2(before - e[0]).unsqueeze(-1)
        codes[slots] = x / torch.exp2(e[index]).unsqueeze(-1)
        scales[of] = (e + 127).to(torch.uint8)
    return {"codes": codes, "scales": scales}


def _exact_verify(c, s):
    B, T, V = c["B"], c["T"], c["V"]
    tokens, paths, counts = [], [], []
    for b, n in enumerate(s["lens"].tolist()):
        x, u = s["tokens"][b].tolist(), s["uniform"][b].double().tolist()
        lines = [(2 << t) - 1 for t in range(T)] if s["tree_mask"] is None else s["tree_mask"][b].tolist()
        above = [max([j for j in range(t) if lines[t] >> j & 1], default=-1) for t in range(T)]
        path, gone = [0], []
        while True:
            p = s["probs"][b, path[-1]].double()
            gone, rest, next_node = [], 1.0, None
            for t in [t for t in range(1, n) if above[t] == path[-1]]:
                w = 0.0 if x[t] in gone else float(p[x[t]])
                share = rest if s["draft_probs"] is None else float(s["draft_probs"][b, t - 1, x[t]])
                if u[t] * share < w:
                    next_node = t
                    break
                rest -= w
                gone.append(x[t])
            if next_node is None:
                break
            path.append(next_node)
        w = p.clone()
        if gone and s["draft_probs"] is not None:
            w = torch.relu(p - s["draft_probs"][b, path[-1]].double())
        elif gone:
            w[gone] = 0
        w = p if float(w.sum()) == 0 else w
        run = torch.cumsum(w, 0)
        above_mark = run > u[0] * run[-1]
        new = int(above_mark.int().argmax())
        tokens.append([x[t] for t in path[1:]] + [new] + [-1] * (T - len(path)))
        paths.append(path + [-1] * (T - len(path)))
        counts.append(len(path))
    return {k: torch.tensor(v, dtype=torch.int32) for k, v in (("tokens", tokens), ("path", paths), ("counts", counts))}


def _exact_pages(c, s):
    kind, page, P = c["kind"], c["page"], c["P"]
    refs, table = s["refs"].tolist(), s["table"].tolist()
    if kind == "copy":
        pairs = list(zip(s["src"].tolist(), s["dst"].tolist()))
    elif kind == "free":
        for row, n in zip(table, s["lens"].tolist()):
            for j in range(-(-n // page), c["M"]):
                if row[j] >= 0:
                    refs[row[j]] -= 1
                    row[j] = -1
        return {"refs": torch.tensor(refs, dtype=torch.int32), "table": torch.tensor(table, dtype=torch.int32)}
    elif kind == "extend":
        free, lacking = iter([i for i in range(P) if refs[i] <= 0]), []
        for row, n in zip(table, s["lens"].tolist()):
            short = 0
            for j in range(min(-(-n // page), c["M"])):
                if row[j] < 0:
                    row[j] = next(free, -1)
                    short += row[j] < 0
                    if row[j] >= 0:
                        refs[row[j]] = 1
            lacking.append(short)
        return {"refs": torch.tensor(refs, dtype=torch.int32), "table": torch.tensor(table, dtype=torch.int32),
                "lacking": torch.tensor(lacking, dtype=torch.int32)}
    elif kind == "fork":
        free, lacking, pairs, child = iter([i for i in range(P) if refs[i] <= 0]), [], [], []
        lens = s["lens"].tolist()
        for parent in s["parents"].tolist():
            row, full = [-1] * c["M"], lens[parent] // page
            for j in range(full):
                row[j] = table[parent][j]
                if row[j] >= 0:
                    refs[row[j]] += 1
            short = 0
            if lens[parent] % page and table[parent][full] >= 0:
                row[full] = next(free, -1)
                short = int(row[full] < 0)
                if not short:
                    refs[row[full]] = 1
                    pairs.append((table[parent][full], row[full]))
            child.append(row)
            lacking.append(short)
    else:
        n = sum(r > 0 for r in refs)
        pairs = list(zip([i for i in range(n, P) if refs[i] > 0], [i for i in range(n) if refs[i] <= 0]))
        to = dict(pairs)
        moved = [to.get(i, i) if refs[i] > 0 else -1 for i in range(P)]
        table = [[moved[e] if e >= 0 else e for e in row] for row in table]
        for a, b in pairs:
            refs[b], refs[a] = refs[a], 0
    buffers = [buffer.clone() for buffer in s["buffers"]]
    if pairs:
        src, dst = torch.tensor(pairs, device="cuda").t()
        for buffer, old in zip(buffers, s["buffers"]):
            buffer.view(P, -1)[dst] = old.view(P, -1)[src]
    if kind == "copy":
        return buffers
    refs = torch.tensor(refs, dtype=torch.int32)
    if kind == "fork":
        return {"refs": refs, "child": torch.tensor(child, dtype=torch.int32), "lacking": torch.tensor(lacking, dtype=torch.int32),
                "buffers": buffers}
    return {"refs": refs, "table": torch.tensor(table, dtype=torch.int32), "moved": torch.tensor(moved, dtype=torch.int32),
            "buffers": buffers}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("write", "keep"):
        return _exact_store(case, s)
    return {"attend": _exact_attend, "verify": _exact_verify, "pages": _exact_pages}[case["op"]](case, s)
