"""The example layer against its float64 form over the keys and values that its cache holds.

With the cache's own values on both sides its width does not enter, and what is left is rounding to bf16: the queries'
(2^-9 of each element at most, so scores of a few units move by under 0.3%), the attention result's (2^-9, 0.17% rms)
and what follows from it in the output product.  1% is allowed at both widths; a lost factor, a wrong position or
one position too many moves results by more.
"""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

from post_weight_quantization_gptq_amd import Context  # noqa: E402

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_step.py")
    spec = importlib.util.spec_from_file_location("draft_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def weights(m, p):
    s, z = (t.double().repeat_interleave(m.GROUP, 1) for t in (p["scales"], p["zeros"]))
    return (s * (p["codes"].double() - z)).to(torch.bfloat16).double()


def over_the_cache(m, layer, x, b, positions, see):
    """Outputs in float64 of tokens x [tokens, HIDDEN] of sequence b, see [tokens, positions of its cache]."""
    n = see.shape[1]
    rows = (x.double() @ weights(m, layer.qkv).T).view(x.shape[0], -1, m.DIM)
    cos, sin = (t[:, None] for t in layer.table.double()[positions].unbind(1))
    a, c = rows[:, :m.HEADS, :m.DIM // 2], rows[:, :m.HEADS, m.DIM // 2:]
    q = torch.cat([a * cos - c * sin, c * cos + a * sin], -1)
    at = torch.arange(n, device=x.device)
    slots = (layer.pages[b][at // layer.page] * layer.page + at % layer.page).to(torch.int32)
    k, v = (t.double().repeat_interleave(m.HEADS // m.KV_HEADS, 1) for t in layer.ctx.kv_read(layer.cache, slots, torch.float32))
    s = torch.matmul(q.transpose(0, 1), k.permute(1, 2, 0).contiguous()) / m.DIM ** 0.5
    p = torch.softmax(s.masked_fill(~see, float("-inf")), -1)
    o = torch.matmul(p, v.transpose(0, 1).contiguous()).transpose(0, 1).reshape(-1, m.HEADS * m.DIM)
    return o @ weights(m, layer.o).T


@pytest.mark.parametrize("bits", [4, 8])
def test_draft_step_over_its_cache(bits):
    m = example()
    prompt, draft = 150, 7
    parents = [-1, 0, 0, 1, 1, 2, 5]
    words, depth = [], []
    for i, p in enumerate(parents):
        words.append((0 if p < 0 else words[p]) | 1 << i)
        depth.append(0 if p < 0 else depth[p] + 1)
    see = torch.ones((draft, prompt + draft), dtype=torch.bool)
    see[:, prompt:] = torch.tensor([[bool(w >> j & 1) for j in range(draft)] for w in words])
    g = torch.Generator().manual_seed(2)
    x = torch.randn((2, prompt + draft, m.HIDDEN), generator=g).to(torch.bfloat16).cuda()
    with Context() as ctx:
        layer = m.Layer(ctx, 2, 256, bits)
        none = torch.zeros(2, dtype=torch.int32, device="cuda")
        pos = torch.arange(prompt, device="cuda").expand(2, -1)
        y = layer(x[:, :prompt], none, pos)
        for b in range(2):
            chain = torch.ones((prompt, prompt), dtype=torch.bool, device="cuda").tril()
            ref = over_the_cache(m, layer, x[b, :prompt], b, pos[b], chain)
            err = float((y[b].double() - ref).norm() / ref.norm())
            print("prompt: error %.2e" % err, flush=True)
            assert 0 < err <= 0.01
        at = prompt + torch.tensor(depth, device="cuda").expand(2, -1)
        mask = torch.tensor(words, dtype=torch.int32, device="cuda").view(1, draft, 1).repeat(2, 1, 1)
        y = layer(x[:, prompt:], none + prompt, at, mask)
        for b in range(2):
            ref = over_the_cache(m, layer, x[b, prompt:], b, at[b], see.cuda())
            err = float((y[b].double() - ref).norm() / ref.norm())
            print("draft: error %.2e" % err, flush=True)
            assert 0 < err <= 0.01
            for t in range(draft):  # without what a token sees of the draft, the same reference is further away
                less = see.clone()
                less[t, prompt + t] = False
                other = over_the_cache(m, layer, x[b, prompt:], b, at[b], less.cuda())[t]
                assert float((y[b, t].double() - other).norm()) > float((y[b, t].double() - ref[t]).norm())
