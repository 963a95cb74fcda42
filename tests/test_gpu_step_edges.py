"""A served step on the GPU where a hand-over, a border, a size or a rounding decides the result."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import step_ref  # noqa: E402
import post_weight_quantization_gptq_amd as gptq  # noqa: E402
from post_weight_quantization_gptq_amd import Adapters, Context, GPTQError  # noqa: E402
from test_gpu_step import (Tables, adapters_of, check_adapters, check_probabilities, check_verify,  # noqa: E402
                           draft_case, f32, i32, layer, rows_of, up)

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ctx():
    c = Context("cuda:0")
    yield c
    c.close()


# --------------------------------------------------------- verification --
def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def long_walk(g, tokens, vocab, rejected):
    """One sequence whose walk accepts every node but those of `rejected`, which have the next node as their sibling.

    A rejected node's token is the one of the largest q - p (its test is 0.999 q < p: false), its sibling's that of the
    largest p - q, of which max(p - q, 0) leaves something; every other node is a child of the last accepted one and
    tested with 0 < p."""
    p = softmax(g.standard_normal((1, tokens, vocab)))
    q = softmax(g.standard_normal((1, tokens, vocab)))
    draft, parents, u = np.zeros((1, tokens), np.int64), np.full((1, tokens), -1), np.zeros((1, tokens), np.float32)
    last = 0
    for i in range(1, tokens):
        parents[0, i] = last
        d = p[0, last].astype(np.float64) - q[0, last]
        if i in rejected:
            draft[0, i], u[0, i] = np.argmin(d), 0.999
        else:
            draft[0, i] = np.argmax(d)
            last = i
    u[0, 0] = 0.6
    return dict(p=p, q=q, draft=draft, parents=parents, uniforms=u)


# walks of more than 64 nodes before a sum that another launch adds up, and past the last launch
@pytest.mark.parametrize("tokens,vocab,rejected", [
    (70, 9000, [1, 68]), (140, 8193, [1, 70, 72, 137]), (300, 20001, [65, 67, 130, 195, 260, 297]),
    (520, 8500, [1, 66, 131, 196, 261, 326, 391, 456, 518]), (1024, 12289, [1, 3, 513, 515, 1020, 1022]),
    (200, 9001, [])])
def test_verify_walks_of_more_than_a_wave(ctx, tokens, vocab, rejected):
    c = long_walk(np.random.default_rng(tokens), tokens, vocab, rejected)
    for _ in range(3):
        want = check_verify(ctx, c)
    assert want[1][0] == tokens - len(rejected)


def whole_sum_case(g, seqs, tokens, vocab, empty, drawn):
    """The walk ends at the root, whose children are rejected (of their token p holds nothing)."""
    p, q = (softmax(g.standard_normal((seqs, tokens, vocab))) for _ in range(2))
    if empty:  # the last values, and some whole tiles between, hold nothing
        p[:, :, -empty:] = 0.0
        p[:, :, 4096:8192] = 0.0
    draft = np.zeros((seqs, tokens), np.int64)
    draft[:, 1:] = 5000
    p[:, :, 5000] = 0.0
    parents = np.zeros((seqs, tokens), np.int64)
    parents[:, 0] = -1
    return dict(p=p, q=q if drawn else None, draft=draft, parents=parents if drawn else None)


@pytest.mark.parametrize("seqs,tokens,vocab", [(9, 1, 20000), (9, 2, 20481), (7, 1, 53000), (5, 3, 131072), (3, 2, 270001),
                                               (40, 2, 50003), (260, 1, 24577)])
@pytest.mark.parametrize("empty", [0, 1, 9000])
def test_verify_no_sum_passes_the_whole(ctx, seqs, tokens, vocab, empty):
    """With a random number of 1 or more no sum passes: the last value with r > 0, however the sums round."""
    g = np.random.default_rng(seqs + vocab + empty)
    u = np.full((seqs, tokens), 0.9999, np.float32)
    for drawn in (False, True):
        c = whole_sum_case(g, seqs, tokens, vocab, empty, drawn)
        for u0 in (1.0, 1.5, float("inf"), float("nan"), 1 - 2.0 ** -24, -0.5):
            u[:, 0] = u0
            check_verify(ctx, dict(c, uniforms=u))


def rejected_siblings(g, seqs, tokens, vocab):
    """Trees whose root has all other nodes as children: those of odd sequences are rejected up to a few, those of even
    ones to the last, each by a residual that a sum over the vocabulary gives."""
    p = softmax(g.standard_normal((seqs, tokens, vocab)))
    q = softmax(g.standard_normal((seqs, tokens, vocab)))
    parents = np.zeros((seqs, tokens), np.int64)
    parents[:, 0] = -1
    draft, u = np.zeros((seqs, tokens), np.int64), np.full((seqs, tokens), 0.999, np.float32)
    below = np.argsort(p[:, 0].astype(np.float64) - q[:, 0], -1)
    draft[:, 1:] = below[:, :tokens - 1]
    for b in range(1, seqs, 2):
        draft[b, b % tokens or 1:] = below[b, -1]
    u[:, 0] = g.random(seqs)
    return dict(p=p, q=q, draft=draft, parents=parents, uniforms=u)


# fewer workgroups a sequence than tiles (6 of 13, 1 of 10, 32 of 33, 12 of 32), and sums left to the last one of more
# tiles than it adds at a time
@pytest.mark.parametrize("seqs,tokens,vocab", [(40, 3, 50003), (130, 2, 40001), (257, 2, 9000), (8, 5, 131073), (21, 4, 131072),
                                               (4, 12, 50003), (3, 20, 36864), (2, 11, 69633), (300, 9, 4500)])
def test_verify_several_tiles_a_workgroup(ctx, seqs, tokens, vocab):
    want = check_verify(ctx, rejected_siblings(np.random.default_rng(seqs + vocab), seqs, tokens, vocab))
    assert (want[1][::2] == 1).all()


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("drawn", [True, False])
def test_verify_of_a_served_batch(ctx, tree, drawn):
    check_verify(ctx, draft_case(np.random.default_rng(46), 70, 5, 33001, tree, drawn))


# ------------------------------------------------------- probabilities --
# a row for every kernel: 256 threads; 1024 with 4, 8, 16 and 32 times four values each; block by block
ROWS = [1000, 4096, 16000, 16384, 32768, 50001, 65536, 100003, 131072, 131073, 270001]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", ROWS)
def test_equal_logits_have_equal_probabilities(ctx, vocab, dtype):
    """Wherever they are in the row, the largest in one place."""
    g = torch.Generator().manual_seed(vocab)
    values = torch.randn((9, 7), generator=g).to(dtype)
    values[:, 0] = values.amax(1) + 0.37
    which = torch.randint(1, 7, (9, vocab), generator=g)
    which[torch.arange(9), torch.randint(0, vocab, (9,), generator=g)] = 0
    x = values.gather(1, which)
    p = ctx.probabilities(x.cuda(), torch.linspace(0.3, 2.0, 9).cuda()).cpu()
    for b in range(9):
        for v in range(7):
            assert p[b, which[b] == v].unique().numel() == 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [2, 1000, 20000, 70000, 140000])
def test_probabilities_of_logits_far_apart(ctx, vocab, dtype):
    """Logits whose difference is past the largest number, temperatures that bring it back, and the smallest ones."""
    most = float(torch.finfo(dtype).max)
    x = (torch.linspace(-1, 1, vocab, dtype=torch.float64) * most).to(dtype)[torch.randperm(vocab)]
    x = torch.stack([x, x / 2, x * 2.0 ** -100, x * 2.0 ** -127, x * 0 + most, -x.abs()])[:, None]
    for t in (3.4e38, 1e38, 3e37, 1e36, 1e8, 2.0, 1.9, 1e-30, 1.2e-38, 1e-40):
        temp = torch.full((6,), t)
        check_probabilities(ctx.probabilities(x.cuda(), temp.cuda()), up(x), temp.numpy())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab,seqs", [(2, 20000), (3000, 2000), (20000, 500), (40000, 300), (70000, 200), (140000, 100)])
def test_probabilities_far_below_the_largest(ctx, vocab, seqs, dtype):
    """Rows of two logits, 0 and -d (exact in both types), the others masked: exp(-d / t) / (1 + exp(-d / t)).

    The exponent d log2(e) / t is rounded once, by half a step, 2^-24 of it: d / t times that in the result.  exp2 is within
    2^-23, the sum, the quotient and the product within 2^-24 each: 5 of these, 8 with what is left of higher order."""
    g = torch.Generator().manual_seed(vocab)
    t = torch.exp(8 * torch.rand(seqs, generator=g) - 4)
    d = (t * (15 + 70 * torch.rand(seqs, generator=g))).to(dtype)
    x = torch.full((seqs, 1, vocab), float("-inf"), dtype=dtype)
    places = torch.stack([torch.randperm(vocab, generator=g)[:2] for _ in range(seqs)])
    rows = torch.arange(seqs)
    x[rows, 0, places[:, 0]], x[rows, 0, places[:, 1]] = 0.0, -d
    p = ctx.probabilities(x.cuda(), t.cuda()).cpu()
    s = up(d) / up(t)
    want = np.exp(-s) / (1 + np.exp(-s))
    err = np.abs(up(p[rows, 0, places[:, 1]]) - want) / want / U
    print("largest error %.1f of %.1f" % (err.max(), (s + 8).max()), flush=True)
    assert np.all(err <= s + 8 + 2.0 ** -125 / want / U)
    assert np.all(np.abs(up(p[rows, 0, places[:, 0]]) - 1 / (1 + np.exp(-s))) <= 8 * U)
    assert int((p != 0).sum()) == 2 * seqs


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", ROWS)
def test_probabilities_within_the_roundings(ctx, vocab, dtype):
    """|error| <= p (k d + k E + n + 3 (n / 16 + 4) + 52) 2^-24 + 2^-125, d = (largest - logit) / t, E its mean over p.

    The exponent is rounded once, 2^-24 d of the result, and the difference of two fp32 logits too (k = 2; of two bf16
    ones of these sizes it is exact: k = 1).  exp2 is within 2^-23.  The sum has that of its terms, d on average E; a thread
    adds n of them and makes its sum smaller once for 16 and for each of up to four at the row's end (an exp2 and a
    product, 3; the exponent's parts add up to d); a tree of 10 levels with an exp2, a product and an addition
    each, 4; the quotient and the product."""
    g = torch.Generator().manual_seed(vocab + 1)
    x = (4.0 * torch.randn((4, 2, vocab), generator=g)).to(dtype)
    t = torch.tensor([0.3, 0.77, 1.0, 1.9])
    got, ref = up(ctx.probabilities(x.cuda(), t.cuda())), step_ref.probabilities(up(x), t.numpy())
    d = (up(x).max(-1, keepdims=True) - up(x)) / up(t)[:, None, None]
    k, n = (1 if dtype == torch.bfloat16 else 2), -(-vocab // (256 if vocab <= 4096 else 1024))
    bound = ref * (k * d + k * (ref * d).sum(-1, keepdims=True) + n + 3 * (n / 16 + 4) + 52) * U + 2.0 ** -125
    print("largest error / bound %.3f" % (np.abs(got - ref) / bound).max(), flush=True)
    assert np.all(np.abs(got - ref) <= bound)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", ROWS)
def test_every_value_counts(ctx, vocab, dtype):
    """One logit far above the others at each border of what a workgroup reads at once: its probability is 1, the others'
    are exp(-60); left out of the sum or of the largest value it would be any other number."""
    row = 1024 if vocab <= 4096 else 4096
    at = sorted({v for c in range(0, vocab + row, row) for v in (c - 1, c, c + 1, c + 3, c + 4)} & set(range(vocab)) | {vocab - 1})
    x = torch.zeros((1, len(at), vocab), dtype=dtype, device="cuda:0")
    x[0, torch.arange(len(at)), torch.tensor(at)] = 60.0
    p = ctx.probabilities(x)[0]
    top = p[torch.arange(len(at)), torch.tensor(at)].double()
    assert float((top - 1).abs().max()) <= 8 * U
    low = torch.where(x[0] == 0, p, np.exp(-60)).double()
    assert float((low / np.exp(-60) - 1).abs().max()) <= (60 + 8) * U
    # and one that is not there at all
    x = torch.where(x == 0, 1.0, float("-inf")).to(dtype)
    p = ctx.probabilities(x)[0].double()
    assert bool((p[x[0] == float("-inf")] == 0).all())
    assert float((p[x[0] == 1] * (vocab - 1) - 1).abs().max()) <= (vocab / 256 + 60) * U


def test_probabilities_into_rows_that_overlap(ctx):
    """Refused; sequences and tokens in either order, side by side or apart, are not."""
    x = torch.randn((4, 3, 10), generator=torch.Generator().manual_seed(9)).cuda()
    buf = torch.zeros(1000, device="cuda:0")
    want = ctx.probabilities(x)
    for seq, token in ((30, 10), (10, 40), (31, 10), (100, 33), (11, 44), (10, 45)):
        assert torch.equal(ctx.probabilities(x, out=buf.as_strided((4, 3, 10), (seq, token, 1))), want)
    for seq, token in ((0, 10), (30, 0), (29, 10), (30, 9), (10, 39), (9, 40), (10, 10), (0, 0)):
        with pytest.raises(GPTQError) as e:
            ctx.probabilities(x, out=buf.as_strided((4, 3, 10), (seq, token, 1)))
        assert e.value.status == 1
    assert torch.equal(ctx.probabilities(x[:1], out=buf.as_strided((1, 3, 10), (0, 10, 1))), want[:1])
    assert torch.equal(ctx.probabilities(x[:, :1], out=buf.as_strided((4, 1, 10), (10, 0, 1))), want[:, :1])
    assert torch.equal(ctx.probabilities(x[:1, 0], out=buf.as_strided((1, 10), (3, 1))), want[:1, 0])


# ------------------------------------------------------------- adapters --
# few rows (16, 32, 64, 128, 128 of many outputs), then a size for every tile, 64 x 64 by one and by several workgroups
KERNELS = [(3, 40, 32), (30, 200, 64), (60, 333, 160), (100, 500, 32), (128, 2100, 96), (200, 700, 64), (200, 700, 2048),
           (500, 4090, 1280), (700, 3000, 32), (2000, 3800, 32), (2500, 4000, 32)]


@pytest.mark.parametrize("rank", [8, 16, 32, 72, 128])
@pytest.mark.parametrize("M,N,K", KERNELS)
def test_adapters_in_full(ctx, M, N, K, rank):
    """alpha X down^T enters the second product with all its bits: weights of 0, one rank and one input that are not 0,
    so that Y = alpha up, three exact parts added up, each addition within a step of 2^-23 however it rounds."""
    g = torch.Generator().manual_seed(M + rank)
    count = 31
    X = torch.zeros((M, K), dtype=torch.bfloat16)
    X[:, 5] = 1.0
    down = torch.zeros((count, rank, K), dtype=torch.bfloat16)
    which = torch.arange(count) * 5 % rank
    down[torch.arange(count), which, 5] = 1.0
    upw = torch.randn((count, N, rank), generator=g).to(torch.bfloat16)
    alpha = torch.randn(count, generator=g)
    ids = torch.randint(-1, count, (M,), generator=g, dtype=torch.int32)
    q = torch.zeros((N, K // 8), dtype=torch.int32), torch.zeros((N, 1)), torch.zeros((N, 1), dtype=torch.uint8)
    Y = ctx.gemm_adapters(X.cuda(), *(t.cuda() for t in q), 0, 4, Adapters(down.cuda(), upw.cuda(), alpha.cuda()), ids.cuda())
    a = ids.clamp(min=0).long()
    want = alpha.double()[a, None] * upw.double()[a, :, which[a]] * (ids >= 0)[:, None]
    err = (Y.cpu().double() - want).abs()
    print("largest error %.2f of 6" % float((err / want.abs().clamp(min=1e-30)).max() / U), flush=True)
    assert bool((err <= 6 * U * want.abs()).all())


LARGE = KERNELS[7:]  # 128 x 128 by two workgroups and by one, 128 x 256, 256 x 256


@pytest.mark.parametrize("M,N,K", LARGE)
def test_rows_in_any_order_on_every_tile(ctx, M, N, K):
    """Rows and results of pitched tensors, sixteen rows of an operand with up to as many adapters."""
    q, w = layer(N, K, 32, 4, 5)
    ad, down, upw, alpha = adapters_of(11, 24, K, N, 6)
    wide = torch.full((M, K + 8), float("nan"), dtype=torch.bfloat16)
    wide[:, :K] = rows_of(M, K, 7)
    ids = np.random.default_rng(8).integers(-1, 11, M)
    Y = torch.full((M, N + 3), 7.0, device="cuda:0")
    got = ctx.gemm_adapters(wide.cuda()[:, :K], *q, 32, 4, ad, i32(ids), Y=Y[:, :N])
    assert bool((Y[:, N:] == 7.0).all())
    rows = np.unique(np.r_[0:140, M // 2:M // 2 + 70, M - 70:M])
    check_adapters(got[torch.from_numpy(rows).cuda()], wide[rows, :K], w, down, upw, ids[rows], alpha)


@pytest.mark.parametrize("sort", [False, True])
@pytest.mark.parametrize("M,N,K", LARGE)
def test_an_adapter_reaches_its_own_rows_on_every_tile(ctx, M, N, K, sort):
    """NaN and infinity in one adapter, and in one row of X, change no other row by a bit."""
    q, _ = layer(N, K, 0, 4, 1)
    ad, *_ = adapters_of(5, 24, K, N, 2)
    X = rows_of(M, K, 3).cuda()
    ids = np.random.default_rng(4).integers(-1, 5, M)
    if sort:
        ids.sort()
    mine = np.nonzero(ids == 1)[0]
    row = int(mine[len(mine) // 2])
    want = ctx.gemm_adapters(X, *q, 0, 4, ad, i32(ids))
    ad.down[2, 3, 5], ad.up[2, 7, 1], ad.up[2, 9] = float("nan"), float("inf"), float("nan")
    ad.alpha[2] = float("inf")
    X[row, 17] = float("nan")
    got = ctx.gemm_adapters(X, *q, 0, 4, ad, i32(ids))
    others = torch.from_numpy((ids != 2) & (np.arange(M) != row)).cuda()
    assert torch.equal(got[others], want[others])
    assert bool(got[torch.from_numpy(ids == 2).cuda()].isnan().any(1).all()) and bool(got[row].isnan().all())


@pytest.mark.parametrize("M,N,K", LARGE)
def test_adapters_past_the_largest_bf16_on_every_tile(ctx, M, N, K):
    q, w = layer(N, K, 0, 4, 25)
    X = torch.zeros((M, K), dtype=torch.bfloat16)
    X[:, 0] = 1.0
    down = torch.zeros((2, 8, K), dtype=torch.bfloat16)
    down[:, :, 0] = 1.0
    upw = ((0.5 + torch.rand((2, N, 8), generator=torch.Generator().manual_seed(26))) * 2.0 ** -100).to(torch.bfloat16)
    ids = np.arange(M) % 3 - 1
    got = ctx.gemm_adapters(X.cuda(), *q, 0, 4, Adapters(down.cuda(), upw.cuda(), f32([3.4e38, float("inf")])), i32(ids))
    assert bool(torch.isposinf(got[torch.from_numpy(ids == 1).cuda()]).all())
    rows = np.nonzero(ids != 1)[0][::7]
    check_adapters(got[torch.from_numpy(rows).cuda()], X[rows], w, up(down), up(upw), ids[rows], torch.tensor([3.4e38, 1.0]))


def test_adapters_of_more_outputs_than_a_launch_takes(ctx):
    """Refused before anything is launched."""
    x = torch.zeros(64, dtype=torch.bfloat16, device="cuda:0")
    a, b = gptq._Adapters(None, None, None, 0, 0), x.data_ptr()
    for M, N, K in ((1000, 1 << 26, 0), (200, 1 << 20, 1 << 17), (16384 + 200, 1 << 20, 1 << 17), (2 ** 31 - 1, 1 << 26, 32)):
        with pytest.raises(GPTQError) as e:
            ctx._check(ctx.lib.gptq_gemm_adapters(ctx.handle, b, M, K, b, b, b, N, K, 0, 4, ctypes.byref(a), b, b, N))
        assert e.value.status == 4 and "launch" in str(e.value)


# ------------------------------------------------- the largest of each --
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_probabilities_of_more_rows_than_a_launch_takes(ctx, dtype):
    """2^22 rows and some more, every fourth greedy; one row of 2^22 values."""
    seqs = (1 << 22) + 37
    x = torch.randn((seqs, 5), generator=torch.Generator(device="cuda:0").manual_seed(1), device="cuda:0").to(dtype)
    t = torch.ones(seqs, device="cuda:0")
    t[3::4] = 0.0
    p = ctx.probabilities(x, t).double()
    want = torch.softmax(x.double(), -1)
    first = torch.where(x == x.amax(-1, keepdim=True), torch.arange(5, device="cuda:0"), 5).amin(-1, keepdim=True)
    want[3::4] = (torch.arange(5, device="cuda:0") == first).double()[3::4]
    assert float(((p - want).abs() / want.clamp(min=1e-30)).max()) <= 100 * U
    row = torch.randn((1, 1 << 22), generator=torch.Generator(device="cuda:0").manual_seed(2), device="cuda:0").to(dtype)
    row[0, -1] = 9.0
    p = ctx.probabilities(row).double()
    want = torch.softmax(row.double(), -1)
    assert float(((p - want).abs() / want).max()) <= (4096 * 19 / 16 + 150) * U
    assert int(ctx.probabilities(row, torch.zeros(1, device="cuda:0")).argmax()) == (1 << 22) - 1


def test_verify_of_many_sequences(ctx):
    check_verify(ctx, draft_case(np.random.default_rng(47), 3000, 4, 23, True, True))
    check_verify(ctx, draft_case(np.random.default_rng(48), 700, 3, 8200, False, True))


@pytest.mark.parametrize("seqs,width", [(8192, 5), (8191, 2), (4100, 20)])
def test_tables_of_many_sequences(ctx, seqs, width):
    page = 32
    t = Tables(ctx, seqs * width, seqs, width, page)
    g = np.random.default_rng(seqs)
    lengths = np.zeros(seqs, np.int64)
    for _ in range(3):
        added = g.integers(-3, width * page // 4, seqs)
        _, info = t.extend(lengths, added)
        assert info[1] == 0
        lengths += np.maximum(added, 0)
        rows = g.permutation(seqs)
        t.fork(lengths, rows[:seqs // 2], rows[seqs // 2:2 * (seqs // 2)])
        lengths[rows[seqs // 2:2 * (seqs // 2)]] = lengths[rows[:seqs // 2]]
        t.consistent()
    lengths[::3] = 0
    t.free(lengths)
    t.consistent()
    t.extend(lengths, np.full(seqs, width * page))  # past the tables: nothing changes
    t.consistent()
