"""The serving operators on a quantised key/value cache: their cases, their plain forms and what they have to move.

Four entry points that run between the quantised products of a layer: rotary positions (``rope``), the cache
written and read back on 8- or 4-bit grids (``kv_write``, ``kv_read``) and the attention of one token, a chain or a
tree of drafted tokens over that cache (``tree_attention``).

The cache is paged.  A slot is page * page_size + offset.  Per (token, head) K and V have a grid each, a float32
scale and a uint8 zero point, value = scale * (code - zero).  ``k_codes`` [pages][heads][page_size][bytes] holds a
token's codes side by side (4 bits: code 2i in the low half of byte i, code 2i+1 in the high half); ``v_codes``
[pages][heads][bytes][page_size] holds the tokens of a page side by side (4 bits: byte row j has dimension j in the
low half and j + head_dim/2 in the high half); scales and zeros are [pages][heads][page_size].
"""
import math

import torch

own = False

DEV = "cuda:0"
_context = None


def _library():
    """The library context that a serving program makes once."""
    global _context
    if _context is None:
        from post_weight_quantization_gptq_amd import Context
        _context = Context(DEV)
    return _context


def _kv_cache(s):
    """The cache handle that a serving program makes once from its tensors."""
    if "handle" not in s:
        from post_weight_quantization_gptq_amd import KVCache
        s["handle"] = KVCache(bits=s["bits"], **s["pool"])
    return s["handle"]


DTYPES = {"bf16": torch.bfloat16, "float32": torch.float32}


# ---------------------------------------------------------------- cases --
def listed():
    return [
        # the queries and keys (32 + 8 heads) of four sequences' next token: launch latency
        dict(name="rope_step", op="rope", tokens=4, heads=40, spare=8, dim=128, rot=128, layout="half", dtype="bf16",
             out="bf16", length=8192),
        # a prompt's queries and keys straight from the float32 product, long-context table
        dict(name="rope_prompt", op="rope", tokens=8192, heads=40, spare=8, dim=128, rot=128, layout="half",
             dtype="float32", out="bf16", length=131072),
        # part of each head, adjacent pairs, an odd token count and 12 heads of 64
        dict(name="rope_part", op="rope", tokens=4099, heads=12, spare=0, dim=64, rot=32, layout="interleaved",
             dtype="float32", out="float32", length=8192),
        # one new token for each of 16 sequences: written, and read back
        dict(name="store_step", op="store", seqs=16, tokens=1, heads=8, dim=128, bits=8, page=64, dtype="bf16",
             out="bf16"),
        # two ragged prompts' keys and values from the float32 product into 4 bits, starting inside a page
        dict(name="store_prompt", op="store", seqs=2, tokens=4097, heads=8, dim=128, bits=4, page=64, dtype="float32",
             out="bf16"),
        # the history of four long sequences read back for a dense consumer
        dict(name="read_long", op="read", seqs=4, tokens=8192, heads=8, dim=128, bits=8, page=64, out="bf16"),
        # a short odd history of small heads, 4 bits, float32 out, small pages
        dict(name="read_short", op="read", seqs=3, tokens=101, heads=4, dim=64, bits=4, page=16, out="float32"),
        # one sequence, one token, a short context: latency
        dict(name="attend_one", op="attend", seqs=1, tokens=1, heads=32, kv_heads=8, dim=128, bits=8, page=64,
             context=1000, tree="one"),
        # a served batch, one token each, ragged contexts
        dict(name="attend_batch", op="attend", seqs=32, tokens=1, heads=32, kv_heads=8, dim=128, bits=8, page=64,
             context=8192, tree="one"),
        # trees of 27 drafted tokens in eight sequences, 4-bit cache, one of them without any context
        dict(name="attend_tree", op="attend", seqs=8, tokens=27, heads=32, kv_heads=8, dim=128, bits=4, page=64,
             context=4093, tree="tree"),
        # a chain of five drafted tokens over one very long context, 4 bits
        dict(name="attend_long", op="attend", seqs=1, tokens=5, heads=32, kv_heads=4, dim=128, bits=4, page=128,
             context=131071, tree="chain"),
        # wide trees, a key head for every query head, small pages
        dict(name="attend_wide", op="attend", seqs=4, tokens=64, heads=16, kv_heads=16, dim=64, bits=8, page=16,
             context=2048, tree="tree"),
    ]


def _spread(rng, lo, hi):
    """A whole number in lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "store", "read", "attend", "attend", "attend"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 256])
        rot = rng.choice([dim, dim // 2, dim // 4 // 2 * 2])
        heads = rng.randint(1, 48)
        return dict(op="rope", tokens=_spread(rng, 1, 8192 * 40 * 128 // (heads * dim) // 2), heads=heads,
                    spare=rng.choice([0, 1, 8]), dim=dim, rot=rot, layout=rng.choice(["half", "interleaved"]),
                    dtype=rng.choice(["bf16", "float32"]), out=rng.choice(["bf16", "float32"]),
                    length=_spread(rng, 64, 131072))
    dim, bits, page = rng.choice([64, 96, 128, 192, 256]), rng.choice([4, 8]), rng.choice([16, 32, 64, 128, 256])
    if op in ("store", "read"):
        heads, seqs = rng.randint(1, 16), _spread(rng, 1, 32)
        most = 2 * 4097 * 8 * 128 // (heads * dim * seqs) * (4 if op == "read" else 1)
        c = dict(op=op, seqs=seqs, tokens=_spread(rng, 1, max(1, most)), heads=heads, dim=dim, bits=bits, page=page,
                 out=rng.choice(["bf16", "float32"]))
        if op == "store":
            c["dtype"] = rng.choice(["bf16", "float32"])
        return c
    kv_heads, group, seqs = rng.choice([1, 2, 4, 8]), rng.randint(1, 8), _spread(rng, 1, 32)
    tree = rng.choice(["one", "chain", "tree"])
    tokens = 1 if tree == "one" else _spread(rng, 2, 64)
    # at most the cache of attend_batch, and score rows as many as attend_wide and attend_batch have
    most = min(131072, 32 * 8192 * 8 * 128 // (2 * seqs * kv_heads * dim), 2 ** 25 // (seqs * kv_heads * group * tokens))
    return dict(op="attend", seqs=seqs, tokens=tokens, heads=kv_heads * group, kv_heads=kv_heads, dim=dim, bits=bits,
                page=page, context=_spread(rng, 1, max(2, most)), tree=tree)


# --------------------------------------------------------------- inputs --
def _lengths(case):
    """Tokens that each sequence has before the call: ragged, down to half of the largest; with trees the last
    of several sequences has none."""
    n, most = case["seqs"], case["context"]
    got = [most - (37 * b % n) * most // (2 * n) for b in range(n)]
    if case["tree"] == "tree" and n > 1:
        got[-1] = 0
    return got


def _pool(pages, heads, page, dim, bits, gen):
    """A filled cache: bell-shaped codes round the zero point, scales that differ from token to token."""
    maxq, width = (1 << bits) - 1, dim * bits // 8

    def codes(shape):
        def bell():
            x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
            return x.mul_(maxq / 6).add_(maxq / 2).round_().clamp_(0, maxq).to(torch.uint8)
        return bell() if bits == 8 else bell() | (bell() << 4)

    def scales(top):
        x = torch.randn((pages, heads, page), generator=gen, device=DEV)
        return (0.25 * x).exp_().mul_(top * 6 / maxq)

    def zeros():
        x = torch.randn((pages, heads, page), generator=gen, device=DEV)
        return x.mul_(maxq / 20).add_(maxq / 2).round_().clamp_(0, maxq).to(torch.uint8)

    return dict(k_codes=codes((pages, heads, page, width)), k_scales=scales(1.0), k_zeros=zeros(),
                v_codes=codes((pages, heads, width, page)), v_scales=scales(0.5), v_zeros=zeros())


def _pages(counts, page, gen):
    """A table of page numbers for sequences of `counts` tokens each, pages in random order; -1 where none is."""
    need = [-(-n // page) for n in counts]
    order = torch.randperm(sum(need), generator=gen, device=DEV).to(torch.int32).cpu()
    table, at = torch.full((len(counts), max(need)), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table.to(DEV), sum(need)


def _slots(table, first, tokens, page):
    """The slots of positions first .. first + tokens - 1 of every sequence, int32 [seqs * tokens]."""
    pos = torch.arange(first, first + tokens, device=DEV)
    return (table[:, pos // page] * page + pos % page).reshape(-1).to(torch.int32)


def _tree_mask(case, seed):
    """Ancestor bits of random trees, int32 words [seqs, tokens, words]; the last token of the last tree is a
    place that no draft took: it sees no drafted token, itself included."""
    b, t = case["seqs"], case["tokens"]
    words = -(-t // 32)
    g = torch.Generator().manual_seed(seed)
    see = torch.zeros((b, t, 32 * words), dtype=torch.int64)
    for j in range(t):
        if j:
            parent = (torch.rand(b, generator=g) * j).long()
            see[:, j] = see[torch.arange(b), parent]
        see[:, j, j] = 1
    see[-1, -1] = 0
    bits = (see.reshape(b, t, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).to(torch.int32).to(DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, dim = case["op"], case["dim"]
    if op == "rope":
        # rows of a fused product: the heads to turn, then `spare` heads (the values) that stay
        rows = torch.randn((case["tokens"], case["heads"] + case["spare"], dim), generator=gen, device=DEV)
        x = rows.to(DTYPES[case["dtype"]])[:, :case["heads"]]
        pos = torch.randint(0, case["length"], (case["tokens"],), generator=gen, device=DEV, dtype=torch.int32)
        freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEV) / case["rot"])
        turn = torch.arange(case["length"], dtype=torch.float64, device=DEV)[:, None] * freq
        table = torch.stack([turn.cos(), turn.sin()], 1).float()  # [length, 2, rot / 2]
        return dict(case, x=x, pos=pos, table=table)
    heads, bits, page = case["heads"], case["bits"], case["page"]
    if op in ("store", "read"):
        # a store starts inside a page, a history at its first token
        first = 5 if op == "store" else 0
        table, pages = _pages([first + case["tokens"]] * case["seqs"], page, gen)
        slots = _slots(table, first, case["tokens"], page)
        s = dict(case, slots=slots, pool=_pool(pages, heads, page, dim, bits, gen))
        if op == "store":
            n = case["seqs"] * case["tokens"]
            kv = torch.randn((n, 2 * heads, dim), generator=gen, device=DEV)
            kv *= (0.25 * torch.randn((n, 2 * heads, 1), generator=gen, device=DEV)).exp()
            kv[:, :, ::16] *= 4.0  # the channels that stand out in keys
            kv = kv.to(DTYPES[case["dtype"]])
            s["k"], s["v"] = kv[:, :heads], kv[:, heads:]
        return s
    lengths = _lengths(case)
    table, pages = _pages([n + case["tokens"] for n in lengths], page, gen)
    q = torch.randn((case["seqs"], case["tokens"], heads, dim), generator=gen, device=DEV)
    q *= 2.0 * (0.5 * torch.randn((case["seqs"], case["tokens"], heads, 1), generator=gen, device=DEV)).exp()
    return dict(case, q=q.to(torch.bfloat16), table=table,
                lengths=torch.tensor(lengths, dtype=torch.int32, device=DEV),
                mask=_tree_mask(case, seed) if case["tree"] == "tree" else None,
                pool=_pool(pages, case["kv_heads"], page, dim, bits, gen))


# ---------------------------------------------------------- plain forms --
def _plain_rope(s):
    x, rot = s["x"].float(), s["rot"]
    cos, sin = s["table"][s["pos"].long()].unsqueeze(2).unbind(1)  # [tokens, 1, rot / 2]
    part, rest = x[..., :rot], x[..., rot:]
    if s["layout"] == "half":
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, rest], -1).to(DTYPES[s["out"]])


def _plain_codes(x, bits):
    """Codes, scales and zero points of the rows of x (the last axis) on min-max grids that hold 0."""
    maxq = float((1 << bits) - 1)
    x = x.float()
    lo, hi = x.amin(-1).clamp(max=0.0), x.amax(-1).clamp(min=0.0)
    flat = (hi - lo) < 2.0 ** -100
    scale = torch.where(flat, 1.0, (hi - lo) / maxq)
    inv = 1.0 / scale
    zero = torch.where(flat, 0.0, (-lo * inv).round().clamp(0.0, maxq))
    codes = (x * inv[..., None] + zero[..., None]).round().clamp(0.0, maxq)
    return codes.to(torch.uint8), scale, zero.to(torch.uint8)


def _plain_write(s):
    pool, page, half = s["pool"], s["page"], s["dim"] // 2
    at, off = s["slots"].long() // page, s["slots"].long() % page
    k, pool["k_scales"][at, :, off], pool["k_zeros"][at, :, off] = _plain_codes(s["k"], s["bits"])
    v, pool["v_scales"][at, :, off], pool["v_zeros"][at, :, off] = _plain_codes(s["v"], s["bits"])
    if s["bits"] == 4:
        k = k[..., 0::2] | (k[..., 1::2] << 4)
        v = v[..., :half] | (v[..., half:] << 4)
    pool["k_codes"][at, :, off] = k
    pool["v_codes"][at, :, :, off] = v


def _plain_values(s, at, off):
    """K and V in 32 bits of the tokens at pages `at`, offsets `off`: [..., heads, dim]."""
    pool = s["pool"]
    k, v = pool["k_codes"][at, :, off], pool["v_codes"][at, :, :, off]
    if s["bits"] == 4:
        k = torch.stack([k & 15, k >> 4], -1).flatten(-2)
        v = torch.cat([v & 15, v >> 4], -1)
    k = (k.float() - pool["k_zeros"][at, :, off].float()[..., None]) * pool["k_scales"][at, :, off][..., None]
    v = (v.float() - pool["v_zeros"][at, :, off].float()[..., None]) * pool["v_scales"][at, :, off][..., None]
    return k, v


def _plain_read(s):
    k, v = _plain_values(s, s["slots"].long() // s["page"], s["slots"].long() % s["page"])
    return k.to(DTYPES[s["out"]]), v.to(DTYPES[s["out"]])


def _plain_attend(s):
    b, t, heads, dim = s["q"].shape
    kv_heads, page = s["kv_heads"], s["page"]
    table, lengths = s["table"].long().clamp(min=0), s["lengths"].long()
    pos = torch.arange(table.shape[1] * page, device=DEV)
    k, v = _plain_values(s, table[:, pos // page], (pos % page).expand(b, -1))  # [seqs, positions, heads, dim]
    q = s["q"].float().reshape(b, t, kv_heads, -1, dim).permute(0, 2, 1, 3, 4).flatten(2, 3)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)) * (dim ** -0.5)  # [seqs, kv heads, tokens * group, positions]
    draft = pos - lengths[:, None]  # [seqs, positions]: place among the drafted tokens
    if s["mask"] is None:
        see = draft[:, None, :] <= torch.arange(t, device=DEV)[:, None]
    else:
        place = draft.clamp(0, t - 1)
        word = s["mask"].gather(2, (place // 32)[:, None, :].expand(b, t, -1))
        see = ((word >> (place % 32)[:, None, :]) & 1 == 1) & (draft < t)[:, None, :] | (draft < 0)[:, None, :]
    see = see[:, None, :, None, :]
    scores = scores.view(b, kv_heads, t, -1, pos.numel()).masked_fill(~see, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    o = torch.matmul(p.flatten(2, 3), v.permute(0, 2, 1, 3).contiguous())
    return o.view(b, kv_heads, t, -1, dim).permute(0, 2, 1, 3, 4).reshape(b, t, heads, dim).to(torch.bfloat16)


def run(s):
    op = s["op"]
    if not own:
        if op == "rope":
            return _plain_rope(s)
        if op == "store":
            _plain_write(s)
        return _plain_attend(s) if op == "attend" else _plain_read(s)
    ctx = _library()
    if op == "rope":
        return ctx.rope(s["x"], s["pos"], s["table"], layout=s["layout"], out_dtype=DTYPES[s["out"]])
    cache = _kv_cache(s)
    if op == "store":
        ctx.kv_write(cache, s["k"], s["v"], s["slots"])
    if op in ("store", "read"):
        return ctx.kv_read(cache, s["slots"], dtype=DTYPES[s["out"]])
    return ctx.tree_attention(s["q"], cache, s["table"], s["lengths"], mask=s["mask"])


# ------------------------------------------------------- what it moves --
def work(case):
    op, dim = case["op"], case["dim"]
    size = {"bf16": 2, "float32": 4}
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return dict(bytes=n * dim * (size[case["dtype"]] + size[case["out"]]) + case["tokens"] * (4 * case["rot"] + 4),
                    flops=3 * n * case["rot"])
    row = dim * case["bits"] // 8 + 5  # codes, scale and zero point of one (token, head)
    if op in ("store", "read"):
        n = 2 * case["seqs"] * case["tokens"] * case["heads"]
        if op == "read":
            return dict(bytes=n * (row + dim * size[case["out"]]) + 4 * case["seqs"] * case["tokens"], flops=2 * n * dim)
        return dict(bytes=n * (2 * row + dim * (size[case["dtype"]] + size[case["out"]])) + 8 * case["seqs"] * case["tokens"],
                    flops=8 * n * dim)
    t = case["tokens"]
    held = sum(n + t for n in _lengths(case))
    return dict(bytes=2 * held * case["kv_heads"] * row + 4 * case["seqs"] * t * case["heads"] * dim,
                flops=4 * held * t * case["heads"] * dim)


# --------------------------------------------------------------- exact --
def _exact_grid(x, bits):
    """Values that stand for the rows of x, in 64 bits.  The grid and the rounding to it are float32 steps by
    definition; what a code stands for is not."""
    import numpy as np
    maxq = np.float32((1 << bits) - 1)
    x = x.float().cpu().numpy()
    lo, hi = np.minimum(x.min(-1, keepdims=True), 0), np.maximum(x.max(-1, keepdims=True), 0)
    span = (hi - lo).astype(np.float32)
    flat = span < 2.0 ** -100
    scale = np.where(flat, np.float32(1), span / maxq).astype(np.float32)
    inv = (np.float32(1) / scale).astype(np.float32)
    zero = np.where(flat, np.float32(0), np.clip(np.rint(-lo * inv), 0, maxq)).astype(np.float32)
    codes = np.clip(np.rint(((x * inv).astype(np.float32) + zero).astype(np.float32)), 0, maxq)
    return torch.from_numpy((codes.astype(np.float64) - zero) * scale.astype(np.float64))


def _exact_rows(s, which, slots):
    """The values of `which` ("k" or "v") at `slots` (a flat int64 tensor), in 64 bits: [slots, heads, dim]."""
    pool, page, dim = s["pool"], s["page"], s["dim"]
    codes, n = pool[which + "_codes"], slots.numel()
    if which == "v":
        codes = codes.transpose(2, 3)  # token by token, as the keys
    flat = codes.permute(0, 2, 1, 3).reshape(-1, codes.shape[1], codes.shape[3])[slots].double()
    if s["bits"] == 4:
        high = torch.floor(flat / 16)
        low = flat - 16 * high
        flat = torch.cat([low, high], -1) if which == "v" else torch.stack([low, high], -1).view(n, -1, dim)
    scale, zero = (pool[which + name].permute(0, 2, 1).reshape(-1, codes.shape[1], 1)[slots].double()
                   for name in ("_scales", "_zeros"))
    return scale * flat - scale * zero


def exact(case, seed):
    s = prepare(case, seed)
    op, dim = case["op"], case["dim"]
    if op == "rope":
        x, rot = s["x"].double(), case["rot"]
        rows = s["table"].double()[s["pos"].long()]  # the table is an input, in float32
        z = torch.complex(rows[:, 0], rows[:, 1])[:, None, :]
        got = x.clone()
        first, second = ((slice(0, rot // 2), slice(rot // 2, rot)) if case["layout"] == "half"
                         else (slice(0, rot, 2), slice(1, rot, 2)))
        w = torch.complex(x[..., first], x[..., second]) * z
        got[..., first], got[..., second] = w.real, w.imag
        return got
    if op == "store":
        return _exact_grid(s["k"], case["bits"]), _exact_grid(s["v"], case["bits"])
    if op == "read":
        return _exact_rows(s, "k", s["slots"].long()), _exact_rows(s, "v", s["slots"].long())
    t, page, group = case["tokens"], case["page"], case["heads"] // case["kv_heads"]
    got = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, n in enumerate(_lengths(case)):
        pos = torch.arange(n + t, device=DEV)
        slots = s["table"][b].long()[pos // page] * page + pos % page
        k, v = _exact_rows(s, "k", slots), _exact_rows(s, "v", slots)
        for i in range(t):
            if s["mask"] is None:
                seen = pos <= n + i
            else:
                words = s["mask"][b, i].tolist()
                seen = torch.tensor([True] * n + [bool(words[j // 32] >> (j % 32) & 1) for j in range(t)], device=DEV)
            if not bool(seen.any()):
                continue
            ks, vs = (k, v) if bool(seen.all()) else (k[seen], v[seen])
            q = s["q"][b, i].double().view(case["kv_heads"], group, dim)
            w = torch.softmax(torch.matmul(q, ks.permute(1, 2, 0)) / math.sqrt(dim), -1)
            got[b, i] = torch.matmul(w, vs.permute(1, 0, 2)).reshape(case["heads"], dim)
    return got
