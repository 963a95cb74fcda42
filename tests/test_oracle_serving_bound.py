"""The bound on attention results lets the kernels' own roundings pass and catches coarser ones, CPU only.

An attention in float32 with the kernels' operands (exact code differences, weights times scales as two bfloat16
numbers to nearest, float32 sums) has to lie within oracle.serving_ref.attention_bound; the same with one plausible
loss planted has to exceed it, at every head size and both widths.
"""
import numpy as np
import pytest

from oracle import serving_ref as o

F = np.float32
N, PAGE, TOKENS, HEADS = 192, 32, 8, 4


def case(bits, dim):
    g = np.random.default_rng(100 * bits + dim)
    pool = o.empty_pool(N // PAGE, 1, PAGE, dim, bits)
    k = g.normal(size=(N, 1, dim))
    v = g.normal(size=k.shape) * np.exp(0.7 * g.normal(size=(N, 1, 1))) + 0.3
    o.kv_write(pool, k, v, np.arange(N), bits)
    q = o.bf16(2.0 * g.normal(size=(1, TOKENS, HEADS, dim)))
    return pool, q, np.arange(N // PAGE)[None], [N - TOKENS]


def near(x):
    return o.bf16(x.astype(np.float64)).astype(F)


def cut(x):
    return (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(F)


def rows(pool, bits):
    """(code - zero point, scale) of K and of V, in position order."""
    out = []
    for which in (0, 1):
        codes, scales = [], []
        for j in range(N):
            a, at = divmod(j, PAGE)
            name = "kv"[which]
            z = F(pool[name + "_zeros"][a, 0, at])
            codes.append(o.kv_codes(pool, a, 0, at, bits)[which].astype(F) - z)
            scales.append(pool[name + "_scales"][a, 0, at])
        out += [np.array(codes, F), np.array(scales, F)]
    return out


def attention(pool, q, bits, loss=None):
    """float32 with the kernels' operands; loss: what is planted."""
    kc, ks, vc, vs = rows(pool, bits)
    dim = q.shape[-1]
    factor = F(dim ** -0.5 * 1.4426950408889634) * F(1.005 if loss == "scale off by 0.5%" else 1)
    out = np.zeros(q.shape)
    for t in range(q.shape[1]):
        n = N - TOKENS + t + 1
        for h in range(HEADS):
            row = q[0, t, h].astype(F)
            s = (kc[:n] @ row).astype(F) * ks[:n]
            if loss == "scores in bf16":
                s = near(s)
            if loss == "scales of the keys in bf16":
                s = (kc[:n] @ row).astype(F) * near(ks[:n])
            if loss == "a position's scale for the next":
                s = (kc[:n] @ row).astype(F) * np.roll(ks[:n], 1)
            e = np.exp2((s * factor - s.max() * factor).astype(F)).astype(F)
            w = (e * vs[:n]).astype(F)
            lead = cut(w) if loss == "weights in one cut bf16" else near(w)
            rest = near(w - lead) if loss not in ("weights in one bf16", "weights in one cut bf16") else np.zeros_like(w)
            acc = (lead @ vc[:n] + rest @ vc[:n]).astype(F)
            total = e[1:].sum(dtype=F) if loss == "a weight not summed" else e.sum(dtype=F)
            out[0, t, h] = acc / total
    return o.bf16(out)


def ratio(bits, dim, loss=None):
    pool, q, tables, lengths = case(bits, dim)
    ref, spread, top = o.tree_attention(q, pool, tables, lengths, bits)
    return float((np.abs(attention(pool, q, bits, loss) - ref) / o.attention_bound(ref, spread, top, dim)).max())


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_the_operands_own_roundings_pass(bits, dim):
    assert ratio(bits, dim) <= 1.0


LOSSES = ["weights in one bf16", "weights in one cut bf16", "scores in bf16",
          "scales of the keys in bf16", "scale off by 0.5%", "a position's scale for the next", "a weight not summed"]


@pytest.mark.parametrize("loss", LOSSES)
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
def test_a_coarser_result_is_caught(bits, dim, loss):
    assert ratio(bits, dim, loss) > 1.0


def test_rounding_to_bf16():
    assert [float(o.bf16(np.float64(x))) for x in (1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -1 - 2.0 ** -8 - 2.0 ** -40, 0.0)] == [
        1.0, 1.0, 1 + 2.0 ** -6, -1 - 2.0 ** -7, 0.0]
