"""The serving operators on the GPU against their float64 oracle.

Rotary results: two products and a sum in float32, |error| <= 3 u (|a c| + |b s|)
with u = 2^-24, and half a bf16 spacing (2^-8 |y|) more where the result is
rounded to bf16.  Codes, scales and zero points come from the same float32 steps
on both sides and are equal.  Attention results: oracle.attention_bound, derived
from the operands' widths.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import serving_ref as o  # noqa: E402
from post_weight_quantization_gptq_amd import Context, GPTQError, KVCache  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ctx():
    c = Context("cuda:0")
    yield c
    c.close()


def up(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda:0")


# --------------------------------------------------------------- rotary --
SCALINGS = [None, dict(kind="linear", factor=4.0), dict(kind="base", factor=8.0),
            dict(kind="parts", factor=4.0, original=64, low=1.0, high=4.0, magnitude=1.2)]


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("length,rot", [(1, 2), (300, 64), (77, 50)])
def test_rope_table(ctx, scaling, length, rot):
    if rot == 2 and scaling and scaling["kind"] == "base":
        with pytest.raises(GPTQError):
            ctx.rope_table(length, rot, scaling=scaling)
        return
    got = up(ctx.rope_table(length, rot, 500.0, scaling))
    ref = o.rope_table(length, rot, 500.0, scaling)
    assert got.shape == ref.shape
    # one rounding to float32, and angles of up to 300 in float64
    assert np.all(np.abs(got - ref) <= U * np.abs(ref) + 1e-12)


def test_rope_table_far_positions(ctx):
    n = 1 << 20
    got = up(ctx.rope_table(n, 8)[-3:])
    w = o.rope_frequencies(8)
    for r, p in enumerate(range(n - 3, n)):
        assert np.abs(got[r, 0] - np.cos(p * w)).max() <= U + 1e-9
        assert np.abs(got[r, 1] - np.sin(p * w)).max() <= U + 1e-9


def rope_error(y, x, pos, table, layout, inverse, bf16):
    ref = o.rope(x, pos, table, layout, inverse)
    mag = o.rope(np.abs(x), pos, np.abs(table), layout, True)  # a c + b s on one side of each pair ...
    mag = np.maximum(mag, o.rope(np.abs(x), pos, np.abs(table), layout, False))  # ... and on the other
    tol = 3 * U * mag + (2.0 ** -8 * np.abs(ref) if bf16 else 0.0) + 1e-37
    rot = 2 * table.shape[2]
    if not bf16:
        assert np.array_equal(y[..., rot:], ref[..., rot:])
    return np.abs(y - ref), tol


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tin,tout", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(1, 1, 64, 64), (7, 5, 80, 20), (3, 40, 128, 128), (33, 3, 96, 48),
                                                  (5, 2, 10, 6), (300, 9, 256, 64), (2, 3, 64, 0)])
def test_rope(ctx, layout, tin, tout, tokens, heads, dim, rot):
    g = np.random.default_rng(tokens * dim + rot)
    x = torch.from_numpy(g.normal(size=(tokens, heads + 2, dim))).to(DTYPES[tin]).cuda()
    view = x[:, 1:1 + heads]  # heads inside a wider row
    pos = g.integers(0, 50, tokens)
    table = ctx.rope_table(50, rot)
    y = ctx.rope(view, i32(pos), table, layout, out_dtype=DTYPES[tout])
    assert y.dtype == DTYPES[tout] and y.shape == view.shape
    err, tol = rope_error(up(y), up(view), pos, up(table), layout, False, tout == "bf16")
    assert np.all(err <= tol)
    z = ctx.rope(view, i32(pos), table, layout, inverse=True, out_dtype=DTYPES[tout])
    err, tol = rope_error(up(z), up(view), pos, up(table), layout, True, tout == "bf16")
    assert np.all(err <= tol)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_in_place_and_into_a_view(ctx, layout):
    g = torch.Generator().manual_seed(3)
    x = torch.randn((21, 6, 64), generator=g).cuda()
    pos, table = i32(np.arange(21)), ctx.rope_table(64, 32)
    want = ctx.rope(x, pos, table, layout)
    wide = torch.full((21, 9, 64), 7.0, device="cuda:0")
    ctx.rope(x, pos, table, layout, out=wide[:, 2:8])
    assert torch.equal(wide[:, 2:8], want) and bool((wide[:, :2] == 7).all()) and bool((wide[:, 8:] == 7).all())
    assert ctx.rope(x, pos, table, layout, out=x) is x
    assert torch.equal(x, want)


def test_rope_odd_alignment(ctx):
    """Rows that start on odd addresses and strides."""
    g = torch.Generator().manual_seed(4)
    flat = torch.randn(5 * 203 + 1, generator=g).to(torch.bfloat16).cuda()
    view = flat[1:].as_strided((5, 3, 66), (203, 67, 1), 1)
    pos, table = i32([0, 5, 3, 9, 2]), ctx.rope_table(10, 34)
    for layout in ("half", "interleaved"):
        y = ctx.rope(view, pos, table, layout, out_dtype=torch.float32)
        assert torch.equal(y, ctx.rope(view.contiguous(), pos, table, layout, out_dtype=torch.float32))
        err, tol = rope_error(up(y), up(view), [0, 5, 3, 9, 2], up(table), layout, False, False)
        assert np.all(err <= tol)


def test_rope_positions_outside_the_table(ctx):
    x = torch.ones((4, 2, 16), device="cuda:0")
    y = ctx.rope(x, i32([0, -1, 10, 2 ** 31 - 1]), ctx.rope_table(10, 8))
    assert bool(y[0].isfinite().all()) and bool(y[1:, :, :8].isnan().all()) and bool((y[1:, :, 8:] == 1).all())


def test_rope_refusals(ctx):
    x, pos, table = torch.zeros((2, 3, 16), device="cuda:0"), i32([0, 1]), ctx.rope_table(4, 8)
    for call in (lambda: ctx.rope(x[0], pos, table), lambda: ctx.rope(x, pos[:1], table),
                 lambda: ctx.rope(x, pos, table, layout="other"), lambda: ctx.rope(x.cpu(), pos, table),
                 lambda: ctx.rope(x, pos, ctx.rope_table(4, 18)), lambda: ctx.rope(x, pos, table, out=x[:, :2]),
                 lambda: ctx.rope(x.transpose(1, 2), pos, table)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ctx.rope(x.half(), pos, table), lambda: ctx.rope(x, pos.long(), table),
                 lambda: ctx.rope(x, pos, table, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: ctx.rope_table(4, 7), lambda: ctx.rope_table(4, 8, base=-1.0), lambda: ctx.rope_table(4, 258),
                 lambda: ctx.rope_table(4, 8, scaling=dict(kind="linear", factor=0.0)),
                 lambda: ctx.rope_table(4, 8, scaling=dict(kind="parts", factor=2.0)),
                 lambda: ctx.rope(x[:, :, :15], pos, table)):
        with pytest.raises(GPTQError):
            call()
    with pytest.raises(ValueError):
        ctx.rope_table(4, 8, scaling=dict(kind="other"))
    assert ctx.rope(x[:0], pos[:0], table).shape == (0, 3, 16)
    assert ctx.rope(x[:, :0], pos, table).shape == (2, 0, 16)


# ---------------------------------------------------------------- cache --
def host_pool(cache):
    return {n: getattr(cache, n).cpu().numpy() for n in KVCache.FIELDS}


def fill(cache, value=0xA5):
    for n in KVCache.FIELDS:
        getattr(cache, n).fill_(float("nan") if n.endswith("scales") else value)


def some_rows(g, tokens, heads, dim):
    x = g.normal(size=(tokens, heads, dim)) * np.exp(g.normal(size=(tokens, heads, 1)))
    x[:, :, ::16] *= 5
    if tokens > 6:
        x[1, 0] = np.abs(x[1, 0])
        x[2, 0] = -np.abs(x[2, 0])
        x[3, 0] = 0.0
        x[4, 0] *= 1e-34  # below the smallest range that is held
        x[5, 0, dim - 1] = np.inf
        x[6, 0, 3] = np.nan
    return x


def run_slots(g, kind, tokens, page, pages):
    if kind == "run":  # positions 5.. of one sequence, pages in any order
        order = g.permutation(pages)
        p = 5 + np.arange(tokens)
        return order[p // page] * page + p % page
    s = g.permutation(pages * page)[:tokens]
    if tokens > 4:
        s[tokens // 2] = -1
        s[0] = pages * page
    return s


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("tokens,heads,dim,page,kind", [
    (1, 1, 64, 16, "any"), (1, 8, 128, 64, "any"), (16, 3, 96, 32, "any"), (63, 2, 128, 16, "run"),
    (64, 1, 192, 128, "run"), (65, 2, 256, 64, "any"), (130, 2, 64, 256, "run"), (201, 1, 96, 16, "run")])
def test_kv_write_and_read(ctx, dtype, bits, tokens, heads, dim, page, kind):
    g = np.random.default_rng(tokens + dim + bits)
    pages = (tokens + 5) // page + 2
    x = torch.from_numpy(some_rows(g, tokens, 2 * heads + 1, dim)).to(DTYPES[dtype]).cuda()
    k, v = x[:, :heads], x[:, heads:2 * heads]  # inside a fused row
    slots = run_slots(g, kind, tokens, page, pages)
    cache = ctx.kv_cache(pages, heads, dim, bits, page)
    fill(cache)
    want = host_pool(cache)
    ctx.kv_write(cache, k, v, i32(slots))
    o.kv_write(want, k.float().cpu().numpy(), v.float().cpu().numpy(), slots, bits)
    got = host_pool(cache)
    for n in KVCache.FIELDS:
        assert np.array_equal(got[n], want[n], equal_nan=n.endswith("scales")), n
    kr, vr = o.kv_read(want, slots, bits)
    for out in (torch.float32, torch.bfloat16):
        a, b = ctx.kv_read(cache, i32(slots), dtype=out)
        for x, r in ((a, kr), (b, vr)):
            r = torch.from_numpy(r).to(out)
            assert x.dtype == out and torch.equal(torch.nan_to_num(x.cpu(), nan=123.0), torch.nan_to_num(r, nan=123.0))
    wide = torch.full((tokens, 2 * heads + 1, dim), 3.0, device="cuda:0")
    ctx.kv_read(cache, i32(slots), k=wide[:, 1:1 + heads], v=wide[:, 1 + heads:])
    assert bool((wide[:, 0] == 3).all())
    assert torch.equal(wide[:, 1:1 + heads].nan_to_num(9.0), torch.from_numpy(kr).cuda().nan_to_num(9.0))
    assert torch.equal(wide[:, 1 + heads:].nan_to_num(9.0), torch.from_numpy(vr).cuda().nan_to_num(9.0))


def test_k_rows_are_packed_rows(ctx):
    """A token's keys in a 4-bit cache are what pack_codes makes of their codes."""
    x = torch.randn((1, 1, 64), generator=torch.Generator().manual_seed(5)).cuda()
    cache = ctx.kv_cache(1, 1, 64, 4, 16)
    ctx.kv_write(cache, x, x, i32([3]))
    codes = torch.from_numpy(o.kv_grid(x[0, 0].cpu().numpy(), 4)[2])[None].cuda()
    assert torch.equal(ctx.pack_codes(codes, 4).view(torch.uint8)[0], cache.k_codes[0, 0, 3])


def test_kv_refusals(ctx):
    cache = ctx.kv_cache(2, 2, 64, 8, 16)
    k, s = torch.zeros((3, 2, 64), device="cuda:0"), i32([0, 1, 2])
    for call in (lambda: ctx.kv_write(cache, k[:, :1], k[:, :1], s), lambda: ctx.kv_write(cache, k, k, s[:2]),
                 lambda: ctx.kv_write(cache, k[..., :32], k[..., :32], s), lambda: ctx.kv_write(cache, k, k[:2], s),
                 lambda: ctx.kv_read(cache, s, k=k[:2]), lambda: ctx.kv_read(cache, s[None]),
                 lambda: ctx.kv_cache(2, 2, 80), lambda: ctx.kv_cache(2, 2, 64, 5), lambda: ctx.kv_cache(2, 2, 64, 8, 24)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: ctx.kv_write(cache, k.half(), k.half(), s), lambda: ctx.kv_write(cache, k, k.bfloat16(), s),
                 lambda: ctx.kv_write(cache, k, k, s.long()), lambda: ctx.kv_read(cache, s, dtype=torch.float16),
                 lambda: ctx.kv_write(dict(), k, k, s)):
        with pytest.raises(TypeError):
            call()
    odd = torch.zeros(3 * 2 * 64 + 1, device="cuda:0")[1:].view(3, 2, 64)
    with pytest.raises(GPTQError) as e:
        ctx.kv_write(cache, odd, odd, s)
    assert e.value.status == 4
    parts = {n: getattr(cache, n) for n in KVCache.FIELDS}
    with pytest.raises(ValueError):
        KVCache(bits=4, **dict(parts, v_codes=parts["v_codes"].transpose(2, 3)))
    with pytest.raises(TypeError):
        KVCache(bits=8, **dict(parts, k_zeros=parts["k_scales"]))
    bad = KVCache(bits=4, **parts)  # 64 bytes a row at 4 bits: heads of 128
    assert bad.dim == 128
    a, b = ctx.kv_read(cache, s[:0])
    assert a.shape == (0, 2, 64) and b.shape == (0, 2, 64)
    ctx.kv_write(cache, k[:0], k[:0], s[:0])


# ------------------------------------------------------------ attention --
def tree_mask(g, seqs, tokens):
    """Random trees, int32 words; the last token of the last sequence sees no drafted token."""
    words = (tokens + 31) // 32
    m = np.zeros((seqs, tokens, words), np.uint32)
    for b in range(seqs):
        for t in range(tokens):
            if t:
                m[b, t] = m[b, g.integers(0, t)]
            m[b, t, t // 32] |= np.uint32(1) << np.uint32(t % 32)
    m[-1, -1] = 0
    return m


def attention_case(ctx, g, lengths, tokens, heads, kv_heads, dim, bits, page, mask, sharp=2.0, width=None):
    """A cache written through the library at random pages, everything else in it unwritten (NaN scales)."""
    seqs = len(lengths)
    need = [0 if n < 0 else -(-(n + tokens) // page) for n in lengths]
    pages = sum(need) + 1
    cache = ctx.kv_cache(pages, kv_heads, dim, bits, page)
    fill(cache, 0xFF)
    order, at = g.permutation(pages), 0
    tables = np.full((seqs, max(max(need), 1) if width is None else width), -1, np.int32)
    slots = []
    for b, n in enumerate(need):
        row = order[at:at + n]
        at += n
        tables[b, :min(n, tables.shape[1])] = row[:tables.shape[1]]
        p = np.arange(max(0, lengths[b] + tokens if lengths[b] >= 0 else 0))
        slots.append(row[p // page] * page + p % page if n else p)
    slots = np.concatenate(slots).astype(np.int64)
    k = g.normal(size=(len(slots), kv_heads, dim))
    v = g.normal(size=k.shape) * np.exp(0.7 * g.normal(size=(len(slots), kv_heads, 1))) + 0.3
    if len(slots):
        ctx.kv_write(cache, *(torch.from_numpy(x).float().cuda() for x in (k, v)), i32(slots))
    q = torch.from_numpy(g.normal(size=(seqs, tokens, heads, dim)) * sharp).to(torch.bfloat16).cuda()
    m = None
    if mask == "tree":
        m = tree_mask(g, seqs, tokens)
    return dict(cache=cache, q=q, tables=tables, lengths=np.array(lengths, np.int32), mask=m, bits=bits)


def call(ctx, c, **more):
    m = None if c["mask"] is None else torch.from_numpy(c["mask"].view(np.int32)).cuda()
    return ctx.tree_attention(c["q"], c["cache"], i32(c["tables"]), i32(c["lengths"]), mask=m, **more)


def check(got, c, scale=None):
    ref, spread, top = o.tree_attention(up(c["q"]), host_pool(c["cache"]), c["tables"], c["lengths"], c["bits"],
                                        c["mask"], scale)
    tol = o.attention_bound(ref, spread, top, ref.shape[-1])
    err = np.abs(up(got) - ref)
    print("largest error over its bound %.3f" % (err / tol).max(), flush=True)
    assert np.all(err <= tol)  # NaN fails too


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("lengths,tokens,heads,kv_heads,page,mask", [
    ([0, 1, 70], 1, 2, 1, 16, None),
    ([130], 3, 8, 2, 64, None),
    ([33, 200, 0], 9, 6, 2, 32, "tree"),
])
def test_tree_attention_dims(ctx, bits, dim, lengths, tokens, heads, kv_heads, page, mask):
    g = np.random.default_rng(dim + bits + tokens)
    c = attention_case(ctx, g, lengths, tokens, heads, kv_heads, dim, bits, page, mask)
    check(call(ctx, c), c)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("lengths,tokens,heads,kv_heads,page,mask", [
    ([0], 1, 1, 1, 16, None),            # one position
    ([15, 16, 17, 63, 64, 65, 127, 128, 129], 1, 4, 1, 16, None),
    ([63, 64, -1, 62, 0], 2, 3, 3, 64, "tree"),   # an absent sequence, an empty row
    ([5, 250], 33, 7, 7, 16, "tree"),     # two mask words
    ([100, 3], 64, 4, 2, 128, "tree"),
    ([61], 65, 5, 1, 256, "tree"),        # five query heads a key head, three words
    ([1000, 990], 4, 16, 1, 64, None),
    ([20], 100, 2, 2, 32, None),          # a long chain
    ([4000], 1, 12, 4, 64, None),
])
def test_tree_attention_lengths(ctx, bits, lengths, tokens, heads, kv_heads, page, mask):
    g = np.random.default_rng(sum(lengths) + tokens + bits)
    c = attention_case(ctx, g, lengths, tokens, heads, kv_heads, 64, bits, page, mask)
    got = call(ctx, c)
    check(got, c)
    for b, n in enumerate(lengths):
        if n < 0:
            assert not bool(got[b].any())
    if mask == "tree" and lengths[-1] == 0:
        assert not bool(got[-1, -1].any())
    assert torch.equal(got, call(ctx, c))  # the same bytes again


def test_tree_attention_scale_and_sharp_scores(ctx):
    g = np.random.default_rng(11)
    c = attention_case(ctx, g, [300, 40], 5, 8, 2, 128, 8, 64, "tree", sharp=40.0)
    check(call(ctx, c), c)  # one position takes nearly everything
    check(call(ctx, c, scale=0.0), c, scale=0.0)  # all alike
    check(call(ctx, c, scale=-0.05), c, scale=-0.05)
    c["q"][0, 1] = 0.0
    c["q"][0, 2] *= 1e-30
    check(call(ctx, c), c)


def test_tree_attention_values_of_many_sizes(ctx):
    """Values whose scales differ by 10^6 from token to token, the small ones where the weight is."""
    g = np.random.default_rng(12)
    c = attention_case(ctx, g, [200], 2, 4, 2, 64, 8, 64, None)
    c["cache"].v_scales *= 10.0 ** torch.randint(-6, 1, c["cache"].v_scales.shape,
                                                  generator=torch.Generator().manual_seed(1)).cuda().float()
    check(call(ctx, c), c)


@pytest.mark.parametrize("tokens", [1, 6])
def test_tree_attention_short_tables_and_bad_pages(ctx, tokens):
    """Positions past the table and pages outside the pool are not seen."""
    g = np.random.default_rng(13)
    c = attention_case(ctx, g, [150, 40], tokens, 4, 2, 64, 8, 16, None, width=5)
    check(call(ctx, c), c)
    c["tables"][0, 1] = -1
    c["tables"][0, 3] = c["cache"].pages
    c["tables"][1, :] = -7
    got = call(ctx, c)
    check(got, c)
    assert not bool(got[1].any())
    c["tables"] = np.zeros((2, 0), np.int32)
    assert not bool(call(ctx, c).any())


def test_tree_attention_lengths_past_the_table(ctx):
    """The largest length there is: every position of the table is before the drafted tokens."""
    g = np.random.default_rng(22)
    c = attention_case(ctx, g, [150, 60], 2, 4, 2, 64, 8, 16, None)
    c["tables"] = c["tables"][:, :2].copy()
    c["lengths"] = np.array([2 ** 31 - 1, 2 ** 31 - 2], np.int32)
    check(call(ctx, c), c)


def test_graph_outlives_a_larger_call():
    """A captured call keeps its workspace when a later one needs more."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ctx = Context("cuda:0")
        g = np.random.default_rng(23)
        small = attention_case(ctx, g, [2000], 4, 8, 1, 64, 8, 64, None)
        t, n = i32(small["tables"]), i32(small["lengths"])
        want = ctx.tree_attention(small["q"], small["cache"], t, n)
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = ctx.tree_attention(small["q"], small["cache"], t, n)
        large = attention_case(ctx, g, [3000, 2500], 60, 16, 2, 128, 8, 64, None)
        for _ in range(3):
            call(ctx, large)
            graph.replay()
            side.synchronize()
            assert torch.equal(out, want)
            out.zero_()
        del graph
        ctx.close()


def test_tree_attention_strided_queries_and_output(ctx):
    g = np.random.default_rng(14)
    c = attention_case(ctx, g, [50, 60], 3, 8, 2, 96, 4, 32, None)
    want = call(ctx, c)
    rows = torch.zeros((2, 3, 12, 96), dtype=torch.bfloat16, device="cuda:0")  # a fused row
    rows[:, :, 2:10] = c["q"]
    out = torch.full((2, 3, 10, 96), 5.0, dtype=torch.bfloat16, device="cuda:0")
    c["q"] = rows[:, :, 2:10]
    assert torch.equal(call(ctx, c, out=out[:, :, 1:9]), want)
    assert bool((out[:, :, 0] == 5).all()) and bool((out[:, :, 9] == 5).all())
    c["q"] = rows[:, :, 2:10].transpose(1, 2).contiguous().transpose(1, 2)  # heads outermost
    assert torch.equal(call(ctx, c), want)


def test_tree_attention_not_a_number_stays_in_its_rows(ctx):
    g = np.random.default_rng(15)
    c = attention_case(ctx, g, [70, 30], 2, 4, 2, 64, 8, 16, None)
    want = call(ctx, c)
    q = c["q"].clone()
    c["q"][0, 1, 3, 5] = float("nan")
    got = call(ctx, c)
    assert bool(got[0, 1, 3].isnan().all())
    got[0, 1, 3] = want[0, 1, 3]
    assert torch.equal(got, want)
    c["q"] = q
    a, s = int(c["tables"][1, 0]), 7  # a value row of sequence 1, key head 1
    c["cache"].v_scales[a, 1, s] = float("nan")
    got = call(ctx, c)
    assert bool(got[1, :, 2:].isnan().all())
    got[1, :, 2:] = want[1, :, 2:]
    assert torch.equal(got, want)


def test_tree_attention_long_context(ctx):
    """Many tiles for few rows: the context is split among workgroups and joined."""
    g = np.random.default_rng(16)
    for bits in (8, 4):
        c = attention_case(ctx, g, [9000], 2, 2, 1, 64, bits, 64, None)
        check(call(ctx, c), c)


@pytest.mark.parametrize("tokens,heads", [(1, 2), (3, 40)])
def test_tree_attention_many_ragged_sequences(ctx, tokens, heads):
    """More sequences than a wave has lanes, lengths from none to several shares of the work."""
    g = np.random.default_rng(20)
    lengths = [int(x) for x in g.integers(0, 40, 70)]
    lengths[3], lengths[64], lengths[69], lengths[10] = 3000, 1500, 700, -1
    c = attention_case(ctx, g, lengths, tokens, heads, 2, 64, 8, 16, None)
    check(call(ctx, c), c)


@pytest.mark.parametrize("bits,dim,tokens,heads,kv_heads", [(8, 128, 50, 6, 2), (4, 128, 70, 2, 1), (4, 256, 35, 2, 2),
                                                            (8, 192, 40, 4, 1), (8, 96, 64, 1, 1), (4, 64, 90, 8, 2)])
def test_tree_attention_many_rows(ctx, bits, dim, tokens, heads, kv_heads):
    """49 to 360 rows of a key head, several blocks and shares, a draft that fills whole tiles."""
    g = np.random.default_rng(21 + dim)
    c = attention_case(ctx, g, [700, 0, 130], tokens, heads, kv_heads, dim, bits, 32, "tree")
    check(call(ctx, c), c)
    assert torch.equal(call(ctx, c), call(ctx, c))


def test_tree_attention_offsets_past_32_bits(ctx):
    """A pool of more than 2^32 bytes of codes."""
    pages, heads, dim, page = 17000, 16, 256, 64
    cache = ctx.kv_cache(pages, heads, dim, 8, page)
    assert cache.k_codes.numel() > 2 ** 32
    g = np.random.default_rng(17)
    n = 100
    k = torch.from_numpy(g.normal(size=(n, 2 * heads, dim))).float().cuda()
    tables = np.array([[pages - 1, pages - 3]], np.int32)
    p = np.arange(n)
    slots = i32(tables[0][p // page] * page + p % page)
    ctx.kv_write(cache, k[:, :heads], k[:, heads:], slots)
    a, b = ctx.kv_read(cache, slots, dtype=torch.float32)
    small = ctx.kv_cache(4, heads, dim, 8, page)
    near = np.array([[2, 0]], np.int32)
    there = i32(near[0][p // page] * page + p % page)
    ctx.kv_write(small, k[:, :heads], k[:, heads:], there)
    c, d = ctx.kv_read(small, there, dtype=torch.float32)
    assert torch.equal(a, c) and torch.equal(b, d)
    q = torch.from_numpy(g.normal(size=(1, 1, heads, dim))).to(torch.bfloat16).cuda()
    assert torch.equal(ctx.tree_attention(q, cache, i32(tables), i32([n - 1])),
                       ctx.tree_attention(q, small, i32(near), i32([n - 1])))


def test_tree_attention_refusals(ctx):
    cache = ctx.kv_cache(2, 2, 64, 8, 16)
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16, device="cuda:0")
    t, n = i32([[0], [1]]), i32([3, 4])
    m = torch.zeros((2, 3, 1), dtype=torch.int32, device="cuda:0")
    for f in (lambda: ctx.tree_attention(q[0], cache, t, n), lambda: ctx.tree_attention(q[:, :, :3], cache, t, n),
              lambda: ctx.tree_attention(q[..., :32], cache, t, n), lambda: ctx.tree_attention(q, cache, t[:1], n),
              lambda: ctx.tree_attention(q, cache, t, n[:1]), lambda: ctx.tree_attention(q, cache, t, n, mask=m[:1]),
              lambda: ctx.tree_attention(q, cache, t, n, out=q[:1]), lambda: ctx.tree_attention(q.cpu(), cache, t, n)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: ctx.tree_attention(q.float(), cache, t, n), lambda: ctx.tree_attention(q, cache, t.long(), n),
              lambda: ctx.tree_attention(q, cache, t, n, mask=m.bool())):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: ctx.tree_attention(q, cache, t, n, mask=m[..., :0].contiguous()),
              lambda: ctx.tree_attention(q, cache, t, n, scale=float("inf"))):
        with pytest.raises(GPTQError):
            f()
    assert ctx.tree_attention(q[:, :0], cache, t, n).shape == (2, 0, 4, 64)
    assert ctx.tree_attention(q[:0], cache, t[:0], n[:0]).shape == (0, 3, 4, 64)


# ----------------------------------------------------- streams and graphs --
def test_serving_on_another_stream(ctx):
    """A context on its own stream, called while another stream is current."""
    g = np.random.default_rng(18)
    c = attention_case(ctx, g, [90, 20], 2, 4, 2, 64, 8, 16, None)
    want = call(ctx, c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        own = Context("cuda:0")
    try:
        t, n = i32(c["tables"]), i32(c["lengths"])
        side.wait_stream(torch.cuda.current_stream())
        got = own.tree_attention(c["q"], c["cache"], t, n)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want)
        side.synchronize()
    finally:
        own.close()


def test_serving_in_a_graph():
    """A step (turn, write, attend) captured once and replayed on new inputs, each replay against the eager result."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ctx = Context("cuda:0")
        g = torch.Generator(device="cuda:0").manual_seed(19)
        cache = ctx.kv_cache(40, 2, 64, 8, 16)
        k = torch.randn((600, 2, 64), generator=g, device="cuda:0")
        ctx.kv_write(cache, k, k.flip(0), torch.arange(600, dtype=torch.int32, device="cuda:0"))
        tables = torch.arange(40, dtype=torch.int32, device="cuda:0").view(2, 20)
        table = ctx.rope_table(400, 64)
        qkv = torch.zeros((2, 8, 64), device="cuda:0")
        n, slots = i32([0, 0]), i32([0, 0])

        def step():
            q = ctx.rope(qkv[:, :4], n, table, out_dtype=torch.bfloat16)
            kk = ctx.rope(qkv[:, 4:6], n, table)
            ctx.kv_write(cache, kk, qkv[:, 6:], slots)
            return ctx.tree_attention(q[:, None], cache, tables, n)

        step()
        graph = torch.cuda.CUDAGraph()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = step()
        for i in range(4):
            qkv.copy_(torch.randn(qkv.shape, generator=g, device="cuda:0"))
            n.copy_(i32([200 + 7 * i, 250 + i]))
            slots.copy_(i32([200 + 7 * i, 320 + 250 + i]))
            graph.replay()
            got = out.clone()
            side.synchronize()
            out.zero_()
            assert bool(got.any()) and torch.equal(got, step())
        side.synchronize()
        del graph
        ctx.close()
