"""The decode-step example over a cache held in 4 bits, from tokens to tokens.

Tolerance, as for the layer with a 16-bit cache: about ten roundings of 2^-11 meet in a step's output, whose relative
error in the root mean square stays below 2^-7.  The cache's 4-bit values are no part of that: the layer in 64 bits reads
them as they are, after each new key and value was found within half a step (and 2^-7 of its size, the error of the values
it was coded from) of the one in 64 bits.  Nor is the choice of experts where two of them are as good: the router's scores
are sums over the rounded norm, off by about 2^-11 of a score's size (2, by the router's weights), so a probability by 2^-10
of itself: where the last chosen expert and the first left out differ by less than 2^-9, either is right.
"""
import numpy as np
import pytest

import kv4
from test_gpu_decode_step import dense, example, rms  # noqa: F401  (a fixture)
from test_gpu_sample import answers

pytestmark = pytest.mark.gpu


def reference_step(layer, weights, x, t, got):
    """The step's output in 64 bits; of the right choices of experts the one nearer to `got`."""
    import torch
    L = layer
    wqkv, wo, ups, downs = weights
    b, h, kv, d = L.batch, L.heads, L.kv, L.dim
    qkv = (rms(x) @ wqkv).view(b, h + 2 * kv, d)
    normed = torch.cat([rms(qkv[:, :h]) * L.q_norm.double(), rms(qkv[:, h:h + kv]) * L.k_norm.double()], 1)
    c, s = L.cos_sin[t, :d // 2].double(), L.cos_sin[t, d // 2:].double()
    a, e = normed[..., :d // 2], normed[..., d // 2:]
    turned = torch.cat([a * c - e * s, e * c + a * s], -1)
    codes, params = kv4.read(L.cache, L.page, kv, d, L.group_size, "fp16")
    stands = kv4.values(codes, params)
    at = torch.arange(t + 1, device="cuda")
    pages = L.table.long()[:, at // L.page]  # [b, t + 1]
    k, v = (side[pages, (at % L.page)[None, :]] for side in stands)  # [b, t + 1, kv, d]
    step = params[..., 0].double().repeat_interleave(L.group_size, -1)[:, pages, (at % L.page)[None, :]][:, :, t]
    for new, want, st in ((k[:, t], turned[:, h:], step[0]), (v[:, t], qkv[:, h + kv:], step[1])):
        assert bool(((new - want).abs() <= 0.5 * st + 2.0 ** -7 * want.abs().amax()).all())
    q = turned[:, :h].view(b, kv, h // kv, d)
    p = torch.softmax(torch.einsum("bcgd,btcd->bcgt", q, k) * d ** -0.5, -1)
    mid = x + torch.einsum("bcgt,btcd->bcgd", p, v).reshape(b, h * d) @ wo
    n, E = rms(mid), L.experts
    best, ids = torch.softmax(n @ E.router.double().t(), -1).sort(-1, descending=True)
    out = torch.empty_like(mid)
    for i in range(b):
        choices = [list(range(E.top_k))]
        if E.top_k < E.experts and float(best[i, E.top_k - 1] - best[i, E.top_k]) < 2.0 ** -9:
            choices.append(choices[0][:-1] + [E.top_k])
        rows = []
        for choice in choices:
            y = mid[i].clone()
            for j in choice:
                gu = n[i] @ ups[int(ids[i, j])]
                gate, up = gu[:E.inter], gu[E.inter:]
                y += best[i, j] / best[i, choice].sum() * ((gate * torch.sigmoid(gate) * up) @ downs[int(ids[i, j])])
            rows.append(y)
        out[i] = min(rows, key=lambda y: float((y - got[i]).pow(2).sum()))
    return out


@pytest.mark.parametrize("batch,sizes", [
    (1, dict(hidden=512, heads=4, kv_heads=2, head_dim=64, inter=256, experts=4, top_k=2)),
    (5, dict(hidden=1024, heads=16, kv_heads=2, head_dim=128, inter=512, experts=8, top_k=3)),
])
def test_steps_match_the_layer_in_64_bits(example, batch, sizes):  # noqa: F811
    import torch
    layer = example.Kv4DecodeLayer(batch, 64, seed=3, **sizes)
    weights = [dense(w.words, w.scales) for w in (layer.qkv, layer.o)] + [
        dense(w, s) for w, s in zip(layer.experts.words, layer.experts.scales)]
    g = torch.Generator(device="cuda").manual_seed(9)
    for t in range(20):  # past the first page
        x = torch.randn((batch, layer.hidden), generator=g, device="cuda", dtype=torch.float16)
        got = layer.step(x).double()
        want = reference_step(layer, weights, x.double(), t, got)
        err = (got - want).pow(2).mean().sqrt() / want.pow(2).mean().sqrt()
        assert float(err) < 2.0 ** -7, (t, float(err))
    assert int(layer.status.item()) == 0 and example.w4.w4a16_status(layer.workspace) == 0


def test_a_captured_chain_of_tokens(example):  # noqa: F811
    """Replays of one graph give the tokens of calls one by one, and these are the definition's for the logits at hand."""
    import torch
    kw = dict(hidden=512, heads=8, kv_heads=2, head_dim=64, inter=256, experts=8, top_k=2, vocab=2048, seed=4)
    eager, captured = example.TokenStep(3, 64, **kw), example.TokenStep(3, 64, **kw)
    uniform = torch.rand((12, 3), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    first, u = captured.tokens.clone(), uniform[0].clone()
    captured.step(u)
    captured.layer.lens.zero_()
    captured.tokens.copy_(first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step(u)
    s = eager.sampler
    for t in range(12):
        eager.step(uniform[t])
        u.copy_(uniform[t])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager.tokens, captured.tokens)
        rows = s.logits.double().cpu().numpy()
        for i in range(3):
            right = answers(rows[i], float(uniform[t, i]), *(float(s.settings["temperature"][i]), int(s.settings["top_k"][i]),
                                                            float(s.settings["top_p"][i]), float(s.settings["min_p"][i])))
            assert int(eager.tokens[i]) in right and np.isfinite(float(s.logprobs[i]))
    assert int(s.status.item()) == 0


def test_main_runs(example, capsys):  # noqa: F811
    example.main(["--kv4", "--batch", "2", "--steps", "4", "--hidden", "512", "--inter", "256", "--experts", "4", "--top-k", "2"])
    assert "device status 0" in capsys.readouterr().out
