"""One workspace, zero-filled once, under calls of sizes that come and go as in a server whose batch
changes: every call gives the bits that it gives in a zeroed workspace of its own, and those are the
operator's (the tolerances are those of the operators' own tests)."""
import pytest

from test_gpu_moe_layer import Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import weight_only_int4_03_gb300 as w4
    return w4


@pytest.mark.parametrize("kw", [
    # One token has 16 x 512 gate-up units, more than two for every warp of 152 SMs: some are drawn.
    dict(dtype="fp16", hidden=256, inter=16384, experts=16, top=16),
    dict(dtype="bf16", hidden=512, inter=8192, experts=8, top=2, zeros=True),
    dict(dtype="fp16", hidden=512, inter=256, experts=128, top=8),
], ids=lambda c: f"{c['dtype']}-{c['hidden']}x{c['inter']}-e{c['experts']}")
def test_expert_layer_at_changing_token_counts(w4, kw):
    import torch
    layer = Layer(w4, 31, tokens=64, **kw)
    every = {n: getattr(layer, n) for n in ("x", "residual", "ids", "tw")}
    counts = (1, 8, 9, 64, 4, 33, 12, 16, 1, 3, 64)
    size = lambda t: w4.w4a16_moe_layer_workspace_size(t, kw["hidden"], kw["inter"], kw["experts"], kw["top"])
    shared = torch.zeros(max(map(size, counts)), dtype=torch.uint8, device="cuda")
    for t in counts:
        layer.tokens = t
        for n, v in every.items():
            setattr(layer, n, v[:t])
        layer.ws = torch.zeros(size(t), dtype=torch.uint8, device="cuda")
        layer.y = torch.full_like(layer.x, float("nan"))
        layer.run()
        layer.check()
        alone, layer.ws = layer.y, shared
        for _ in range(2):
            layer.y = torch.full_like(alone, float("nan"))
            layer.run()
            torch.cuda.synchronize()
            assert torch.equal(layer.y, alone), f"{t} tokens"
        assert w4.w4a16_status(shared) == 0
