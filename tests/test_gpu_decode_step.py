"""The decode-step example: the operators together, against the same layer in 64 bits.

Tolerance.  Along the step every product is exact in its inputs and every 16-bit buffer (norms, qkv,
q, attention, projection, middle, output) rounds its values once, a relative error of at most 2^-11
each; the W4A16 products round their weights too, as much again.  About ten such roundings meet in
the output, so its relative error in the root mean square stays below 10 x 2^-11 < 2^-7 a step; the
cache carries earlier steps' errors of the same size.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    import torch
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def dense(words, scales):
    import torch
    q = torch.stack([(words >> (4 * i)) & 15 for i in range(8)], -2).flatten(-3, -2).double()
    return (q - 8) * scales.double().repeat_interleave(128, -2)


def rms(x):
    return x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()


class Reference:
    """The layer from its definition in 64 bits, with a cache of its own."""

    def __init__(self, layer):
        self.layer, self.keys, self.values = layer, [], []
        self.wqkv, self.wo = dense(layer.qkv.words, layer.qkv.scales), dense(layer.o.words, layer.o.scales)
        self.up, self.down = (dense(w, s) for w, s in zip(layer.experts.words, layer.experts.scales))

    def step(self, x):
        import torch
        L = self.layer
        b, h, kv, d = L.batch, L.heads, L.kv, L.dim
        t = len(self.keys)
        qkv = (rms(x) @ self.wqkv).view(b, h + 2 * kv, d)
        c, s = L.cos_sin[t, :d // 2].double(), L.cos_sin[t, d // 2:].double()
        a, e = qkv[:, :h + kv, :d // 2], qkv[:, :h + kv, d // 2:]
        turned = torch.cat([a * c - e * s, e * c + a * s], -1)
        self.keys.append(turned[:, h:])
        self.values.append(qkv[:, h + kv:])
        k, v = torch.stack(self.keys, 1), torch.stack(self.values, 1)  # [b, t, kv, d]
        q = turned[:, :h].view(b, kv, h // kv, d)
        p = torch.softmax(torch.einsum("bcgd,btcd->bcgt", q, k) * d ** -0.5, -1)
        att = torch.einsum("bcgt,btcd->bcgd", p, v).reshape(b, h * d)
        mid = x + att @ self.wo
        n = rms(mid)
        E = L.experts
        probability = torch.softmax(n @ E.router.double().t(), -1)
        best, ids = probability.topk(E.top_k, -1)
        best = best / best.sum(-1, keepdim=True)
        out = mid.clone()
        for i in range(b):
            for j in range(E.top_k):
                e_ = int(ids[i, j])
                gu = n[i] @ self.up[e_]
                gate, up = gu[:E.inter], gu[E.inter:]
                out[i] += best[i, j] * ((gate * torch.sigmoid(gate) * up) @ self.down[e_])
        return out


@pytest.mark.parametrize("batch,sizes", [
    (1, dict(hidden=512, heads=4, kv_heads=2, head_dim=64, inter=256, experts=4, top_k=2)),
    (5, dict(hidden=1024, heads=16, kv_heads=2, head_dim=128, inter=512, experts=8, top_k=3)),
])
def test_steps_match_the_layer_in_64_bits(example, batch, sizes):
    import torch
    layer = example.DecodeLayer(batch, 64, seed=3, **sizes)
    ref = Reference(layer)
    g = torch.Generator(device="cuda").manual_seed(9)
    for t in range(20):  # past the first page
        x = torch.randn((batch, layer.hidden), generator=g, device="cuda", dtype=torch.float16)
        got = layer.step(x).double()
        want = ref.step(x.double())
        err = (got - want).pow(2).mean().sqrt() / want.pow(2).mean().sqrt()
        assert float(err) < 2.0 ** -7, (t, float(err))
    assert int(layer.status.item()) == 0


def test_a_captured_step_serves_every_token(example):
    """Replays of one graph give the same bits as calls one by one."""
    import torch
    kw = dict(hidden=512, heads=8, kv_heads=2, head_dim=64, inter=256, experts=8, top_k=2, seed=4)
    x0 = torch.randn((3, 512), device="cuda", dtype=torch.float16)
    eager, captured = example.DecodeLayer(3, 64, **kw), example.DecodeLayer(3, 64, **kw)
    x, y = x0.clone(), x0.clone()
    captured.step(y)
    captured.lens.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y.copy_(captured.step(y))
    y.copy_(x0)
    for _ in range(12):
        x.copy_(eager.step(x))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, y)


def test_main_runs(example, capsys):
    example.main(["--batch", "2", "--steps", "4", "--hidden", "512", "--inter", "256", "--experts", "4", "--top-k", "2"])
    assert "device status 0" in capsys.readouterr().out


def test_steps_past_the_longest_length_are_reported(example):
    """The cache's end: no page is looked up beyond the table, what is cached stays, and the status words
    tell; up to there a layer with a longer cache gives the same bits."""
    import torch
    kw = dict(hidden=512, heads=4, kv_heads=2, head_dim=64, inter=256, experts=4, top_k=2, seed=5)
    layer, longer = example.DecodeLayer(2, 20, **kw), example.DecodeLayer(2, 80, **kw)
    g = torch.Generator(device="cuda").manual_seed(10)
    for _ in range(20):
        x = torch.randn((2, 512), generator=g, device="cuda", dtype=torch.float16)
        assert torch.equal(layer.step(x), longer.step(x))
    assert int(layer.status.item()) == 0
    caches = layer.k_cache.clone(), layer.v_cache.clone()
    for _ in range(25):
        layer.step(x)
    torch.cuda.synchronize()
    assert torch.equal(layer.k_cache, caches[0]) and torch.equal(layer.v_cache, caches[1])
    assert int(layer.status.item()) == example.w4.W4A16_DEV_POSITION
    assert example.w4.w4a16_status(layer.workspace) == example.w4.W4A16_DEV_LENGTH
    assert example.w4.w4a16_status(longer.workspace) == 0
