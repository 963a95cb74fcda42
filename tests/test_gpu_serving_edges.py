"""Serving operators on the GPU where a rounding, a size or a setting decides the result."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import serving_ref as o  # noqa: E402
from post_weight_quantization_gptq_amd import Context, GPTQError, KVCache  # noqa: E402
from test_gpu_serving import attention_case, call, check, fill, i32, up  # noqa: E402
from test_oracle_serving_grid import PINS  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    c = Context("cuda:0")
    yield c
    c.close()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("tokens,heads,kv_heads", [(1, 4, 1), (5, 8, 1), (32, 2, 1), (60, 4, 2)])
def test_weights_have_no_bias(ctx, bits, tokens, heads, kv_heads):
    """Values that are all the same number, 2^-18 of it above the middle of two bfloat16 numbers, come out as the upper one.

    The result is that number whatever the weights.  About a thousand positions take part with weights of one size, so
    that parts rounded to nearest (each weight within 2^-16, 2^-18.6 rms) leave an error near 2^-23 and float32 sums one
    near 2^-21; parts cut off leave every weight and the result too small by 2^-17.
    """
    g = np.random.default_rng(30 + bits + tokens)
    c = attention_case(ctx, g, [1000, 900], tokens, heads, kv_heads, 64, bits, 32, None, sharp=0.2)
    value = np.float32((1 + 2.0 ** -8) * (1 + 2.0 ** -18))
    cache = c["cache"]
    cache.v_codes.fill_(0x11 if bits == 4 else 1)
    cache.v_zeros.zero_()
    cache.v_scales.fill_(float(value))
    got = call(ctx, c).float()
    assert bool((got == 1 + 2.0 ** -7).all()), "%d of %d results on the lower side" % (int((got < 1.005).sum()), got.numel())


def launched(ctx, names, f):
    """f(), and how often each of the kernels ran in it."""
    ctx.timing(",".join(names))
    try:
        got = f()
        return got, [ctx.kernel_time(n)[1] for n in names]
    finally:
        ctx.timing(None)


@pytest.mark.parametrize("bits,dim", [(8, 64), (4, 96), (8, 96), (4, 128), (8, 192), (4, 192), (8, 256)])
def test_many_shares_are_joined(ctx, bits, dim):
    """More than 16 shares of a row: several threads join each value, at head sizes that do and do not fill a workgroup."""
    g = np.random.default_rng(40 + dim + bits)
    c = attention_case(ctx, g, [4500], 2, 3, 1, dim, bits, 64, None)
    got, (n,) = launched(ctx, ["k_attn_join"], lambda: call(ctx, c))
    assert n == 1
    check(got, c)
    assert torch.equal(got, call(ctx, c))


@pytest.mark.parametrize("mode", ["global", "thread_local", "relaxed"])
def test_a_capture_takes_no_workspace(mode):
    """A call that would have to grow its workspace is refused while its stream is captured; the capture goes on, and the
    same call then runs eagerly and, its workspace there, in a graph."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        own = Context("cuda:0")
        try:
            g = np.random.default_rng(50)
            c = attention_case(own, g, [700, 30], 1, 4, 2, 64, 8, 16, None)  # few shares: joined in the same launch
            t, n = i32(c["tables"]), i32(c["lengths"])
            out = torch.zeros_like(c["q"])
            mark = torch.zeros(1, device="cuda:0")
            side.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side, capture_error_mode=mode):
                mark.add_(1)
                with pytest.raises(GPTQError) as e:
                    own.tree_attention(c["q"], c["cache"], t, n, out=out)
            assert e.value.status == 4 and "capture" in str(e.value)
            graph.replay()
            side.synchronize()
            assert float(mark) == 1 and not bool(out.any())
            want = own.tree_attention(c["q"], c["cache"], t, n)
            check(want, c)
            again = torch.cuda.CUDAGraph()
            side.synchronize()
            with torch.cuda.graph(again, stream=side, capture_error_mode=mode):
                own.tree_attention(c["q"], c["cache"], t, n, out=out)
            for _ in range(3):
                out.zero_()
                again.replay()
                side.synchronize()
                assert torch.equal(out, want) and torch.equal(own.tree_attention(c["q"], c["cache"], t, n), want)
            del graph, again
        finally:
            side.synchronize()
            own.close()


# ---------------------------------------------------- more than one launch --
MANY = (1 << 23) + 100  # tokens of 64 heads: more workgroups of 256 than 2^32 threads make


def test_write_of_more_tokens_than_a_launch_holds(ctx):
    """All tokens are skipped but a few: the first, the last, and those round the end of what one launch can hold."""
    heads, dim, tokens = 64, 64, MANY
    at = [0, 1, 8388000, 8388095, 8388096, 8388097, tokens - 2, tokens - 1]
    x = torch.zeros((tokens, 1, dim), dtype=torch.bfloat16, device="cuda:0")
    x[at] = torch.randn((len(at), 1, dim), generator=torch.Generator().manual_seed(60)).to(torch.bfloat16).cuda()
    slots = torch.full((tokens,), -1, dtype=torch.int32, device="cuda:0")
    slots[at] = i32(range(3, 3 + len(at)))
    few = x[at].expand(-1, heads, -1).contiguous()
    got, want = (ctx.kv_cache(2, heads, dim, 8, 16) for _ in range(2))
    fill(got)
    fill(want)
    ctx.kv_write(got, x.expand(-1, heads, -1), x.flip(2).expand(-1, heads, -1), slots)
    ctx.kv_write(want, few, few.flip(2), i32(range(3, 3 + len(at))))
    for n in KVCache.FIELDS:
        assert torch.equal(getattr(got, n).nan_to_num(7.0), getattr(want, n).nan_to_num(7.0)), n


def test_read_of_more_tokens_than_a_launch_holds(ctx):
    """Heads that hold the same, read into one place: every head writes the same values."""
    heads, dim, tokens = 64, 64, MANY
    cache, one = ctx.kv_cache(4, heads, dim, 8, 16), ctx.kv_cache(4, 1, dim, 8, 16)
    rows = torch.randn((64, 2, dim), generator=torch.Generator().manual_seed(61)).cuda()
    where = torch.arange(64, dtype=torch.int32, device="cuda:0")
    ctx.kv_write(cache, rows[:, :1].expand(-1, heads, -1), rows[:, 1:].expand(-1, heads, -1), where)
    ctx.kv_write(one, rows[:, :1], rows[:, 1:], where)
    slots = torch.randint(-1, 64, (tokens,), generator=torch.Generator().manual_seed(62)).to(torch.int32).cuda()
    k, v = (torch.full((tokens, 1, dim), 9.0, dtype=torch.bfloat16, device="cuda:0") for _ in range(2))
    ctx.kv_read(cache, slots, k=k.expand(-1, heads, -1), v=v.expand(-1, heads, -1))
    for a, b in zip((k, v), ctx.kv_read(one, slots)):
        assert torch.equal(a, b)


def test_rope_table_of_more_values_than_a_launch_holds(ctx):
    """2^32 pairs and some: two launches."""
    length, rot = (1 << 25) + 3, 256
    table = ctx.rope_table(length, rot)
    short = ctx.rope_table(5, rot)
    assert torch.equal(table[:5], short)
    w = o.rope_frequencies(rot)
    for p in ((1 << 24) - 1, 1 << 24, (1 << 24) + 1, (1 << 25) - 1, 1 << 25, length - 1):
        row = up(table[p])  # an angle of 2^25 in float64 is within 2^-28 of its own
        assert np.abs(row[0] - np.cos(p * w)).max() <= 2.0 ** -24 + 1e-8
        assert np.abs(row[1] - np.sin(p * w)).max() <= 2.0 ** -24 + 1e-8


def test_attention_of_more_rows_than_a_launch_holds(ctx):
    """2^24 workgroups are refused before anything is launched."""
    seqs, heads = 1 << 20, 16
    cache = ctx.kv_cache(1, heads, 64, 8, 16)
    q = torch.zeros((1, 1, heads, 64), dtype=torch.bfloat16, device="cuda:0").expand(seqs, -1, -1, -1)
    t, n = torch.zeros((seqs, 1), dtype=torch.int32, device="cuda:0"), torch.zeros(seqs, dtype=torch.int32, device="cuda:0")

    def refused():
        with pytest.raises(GPTQError) as e:
            ctx.tree_attention(q, cache, t, n, out=torch.empty_like(q))
        return e.value

    err, launches = launched(ctx, ["k_tree_attn", "k_tree_attn_wide", "k_attn_join"], refused)
    assert err.status == 4 and "rows" in str(err) and launches == [0, 0, 0]


# ------------------------------------------------------------ score factors --
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("tokens,heads", [(1, 4), (20, 1), (70, 2)])
@pytest.mark.parametrize("queries,keys,scale", [(1e-28, 1e28, None), (1e-33, 1e33, None), (1.0, 1e29, 1e-30),
                                                (1e-5, 1e34, 1e-30), (1e30, 1e-30, None), (1e25, 1e-5, 1e-21)])
def test_factors_far_from_one(ctx, bits, tokens, heads, queries, keys, scale):
    """Queries, keys and a scale far from one whose scores are ordinary."""
    g = np.random.default_rng(70 + bits + tokens)
    c = attention_case(ctx, g, [80, 33], tokens, heads, 1, 64, bits, 16, None)
    c["q"] = (c["q"].float() * queries).to(torch.bfloat16)
    c["cache"].k_scales.mul_(keys)
    check(call(ctx, c, scale=scale), c, scale=scale)


# ------------------------------------------------------------------- handle --
def test_a_cache_keeps_its_tensors(ctx):
    """Other tensors in the place of a cache's are refused, not ignored; the same ones change in place."""
    cache = ctx.kv_cache(2, 1, 64, 8, 16)
    x = torch.randn((3, 1, 64), generator=torch.Generator().manual_seed(80)).cuda()
    ctx.kv_write(cache, x, x, i32([0, 5, 31]))
    k, v = ctx.kv_read(cache, i32([0, 5, 31]), dtype=torch.float32)
    for name in KVCache.FIELDS:
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(cache, name).clone())
    for name, value in (("bits", 4), ("page", 32), ("pages", 9)):
        with pytest.raises(AttributeError):
            setattr(cache, name, value)
    cache.v_scales *= 2.0
    k2, v2 = ctx.kv_read(cache, i32([0, 5, 31]), dtype=torch.float32)
    assert torch.equal(k2, k) and torch.equal(v2, 2 * v)


# ------------------------------------------------------------ every kernel --
def wide(dim, rows):
    """Whether k_tree_attn_wide takes these rows of a key head (tests/attend/check_attend.cpp holds the same table)."""
    return rows == 64 or rows == 128 and dim <= 128


BRANCHES = [(dim, rows) for dim in (64, 96, 128, 192, 256) for rows in ((10, 20, 40, 64, 80, 128) if dim <= 128 else (10, 20, 64, 80))]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim,rows", BRANCHES)
def test_every_attention_kernel(ctx, bits, dim, rows):
    """Each (head size, width, rows a wave, kernel) there is: ragged trees on small pages, and a chain whose context is cut
    into shares, joined by a launch of its own."""
    g = np.random.default_rng(90 + dim + rows + bits)
    names = ["k_tree_attn", "k_tree_attn_wide", "k_attn_join"]
    one = [0, 1] if wide(dim, rows) else [1, 0]
    c = attention_case(ctx, g, [330, 0, 61], rows // 2, 4, 2, dim, bits, 16, "tree")
    got, n = launched(ctx, names, lambda: call(ctx, c))
    assert n[:2] == one
    check(got, c)
    c = attention_case(ctx, g, [4200], rows // 2, 2, 1, dim, bits, 64, None)
    got, n = launched(ctx, names, lambda: call(ctx, c))
    assert n == one + [1]
    check(got, c)
    assert torch.equal(got, call(ctx, c))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_shares_joined_in_the_same_launch(ctx, bits, dim):
    """Up to eight shares of up to 16 rows: the workgroup that comes last joins them, call after call."""
    g = np.random.default_rng(95 + dim + bits)
    c = attention_case(ctx, g, [1900, 700, 0], 2, 6, 2, dim, bits, 32, None)
    got, n = launched(ctx, ["k_tree_attn", "k_attn_join"], lambda: call(ctx, c))
    assert n == [1, 0]
    check(got, c)
    for _ in range(20):
        assert torch.equal(got, call(ctx, c))


# --------------------------------------------------------------------- grid --
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bits,a,zero,codes", PINS)
def test_the_grid_s_step_is_a_product(ctx, dtype, bits, a, zero, codes):
    """Rows on which the product and the quotient by maxq choose different zero points."""
    x = torch.zeros((1, 1, 64), dtype=dtype, device="cuda:0")
    x[0, 0, :3] = torch.tensor([a, -a, a / 2])
    cache = ctx.kv_cache(1, 1, 64, bits, 16)
    ctx.kv_write(cache, x, x, i32([9]))
    s = np.float32(np.float32(2 * a) * np.float32(np.float32(1) / np.float32((1 << bits) - 1)))
    for scales, zeros in ((cache.k_scales, cache.k_zeros), (cache.v_scales, cache.v_zeros)):
        assert float(scales[0, 0, 9]) == float(s) and int(zeros[0, 0, 9]) == zero
    want = np.float32(s) * (np.array(codes, np.float32) - np.float32(zero))
    for r in ctx.kv_read(cache, i32([9]), dtype=torch.float32):
        assert r[0, 0, :3].cpu().numpy().tolist() == want.tolist() and not bool(r[0, 0, 3:].any())


# ---------------------------------------------------------- large results --
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("tin,tout,rot", [(torch.float32, torch.bfloat16, 64), (torch.bfloat16, torch.float32, 128),
                                          (torch.float32, torch.float32, 40), (torch.bfloat16, torch.bfloat16, 128)])
def test_rope_results_past_the_caches(ctx, layout, tin, tout, rot):
    """A result of more than 256 MB is stored another way: the same bytes as in parts."""
    heads, dim = 16, 128
    tokens = (256 << 20) // (heads * dim * torch.finfo(tout).bits // 8) + 77
    x = torch.randn((tokens, heads, dim), generator=torch.Generator(device="cuda:0").manual_seed(85), device="cuda:0").to(tin)
    pos, table = torch.arange(tokens, device="cuda:0").remainder(300).to(torch.int32), ctx.rope_table(300, rot)
    got = ctx.rope(x, pos, table, layout, out_dtype=tout)
    for a in range(0, tokens, tokens // 3):
        b = min(a + tokens // 3, tokens)
        assert torch.equal(got[a:b], ctx.rope(x[a:b], pos[a:b], table, layout, out_dtype=tout))


@pytest.mark.parametrize("bits,dtype", [(8, torch.bfloat16), (4, torch.bfloat16), (4, torch.float32)])
def test_reads_past_the_caches(ctx, bits, dtype):
    heads, dim, page = 4, 128, 64
    tokens = (256 << 20) // (2 * heads * dim * torch.finfo(dtype).bits // 8) + 77
    cache = ctx.kv_cache(40, heads, dim, bits, page)
    x = torch.randn((40 * page, 2 * heads, dim), generator=torch.Generator(device="cuda:0").manual_seed(86), device="cuda:0")
    ctx.kv_write(cache, x[:, :heads], x[:, heads:], torch.arange(40 * page, dtype=torch.int32, device="cuda:0"))
    slots = torch.randint(-1, 40 * page, (tokens,), generator=torch.Generator().manual_seed(87)).to(torch.int32).cuda()
    got = ctx.kv_read(cache, slots, dtype)
    for a in range(0, tokens, tokens // 3):
        b = min(a + tokens // 3, tokens)
        for whole, part in zip(got, ctx.kv_read(cache, slots[a:b], dtype)):
            assert torch.equal(whole[a:b], part)


# ------------------------------------------------------------------ streams --
def test_results_read_on_the_callers_stream(ctx):
    """A context on a stream of its own: memory of a result that the caller's stream has yet to read, freed by the caller,
    is not the next call's result."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        own = Context("cuda:0")
    try:
        here = torch.cuda.current_stream()
        x = torch.randn((4096, 8, 64), generator=torch.Generator().manual_seed(97)).cuda()
        pos, table = i32(np.arange(4096) % 100), own.rope_table(100, 64)
        y, kept, read = -x, torch.empty_like(x), torch.cuda.Event()
        kept.copy_(x)
        side.wait_stream(here)
        a = own.rope(x, pos, table)
        here.wait_stream(side)
        torch.cuda._sleep(50_000_000)  # the caller's stream is some milliseconds behind
        kept.copy_(a)
        read.record(here)
        at = a.data_ptr()
        del a
        b = own.rope(y, pos, table)
        assert b.data_ptr() != at or read.query()  # (a slow host: the read is done)
        here.wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(kept, -b)
    finally:
        torch.cuda.synchronize()
        own.close()
