"""The decode-step example from tokens to tokens: a row that got no token (-1) is looked up as a token that there is."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load():
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_rows_without_a_token_do_not_leave_the_embedding():
    """On the CPU, where an index of -1 is an error and not a fault."""
    import torch
    example = load()
    seen = []

    class Layer:
        def step(self, x):
            seen.append(x.clone())
            return x

    chain = object.__new__(example.TokenStep)
    chain.layer, chain.embedding = Layer(), torch.arange(12.0).view(4, 3)
    chain.tokens = torch.tensor([2, -1, 3], dtype=torch.int32)
    chain.sampler = lambda x, uniform: torch.tensor([1, -1, -1], dtype=torch.int32)
    assert chain.step(None).tolist() == [1, -1, -1]
    assert chain.step(None).tolist() == [1, -1, -1]  # -1 stays to be seen
    assert seen[0][:, 0].tolist() == [6.0, 0.0, 9.0] and seen[1][:, 0].tolist() == [3.0, 0.0, 0.0]


@pytest.mark.gpu
def test_a_row_without_a_token_leaves_the_others_alone():
    """A row with a setting out of range gets -1 at every step, reports it, and the other rows' tokens stay what they were."""
    import torch
    example = load()
    kw = dict(hidden=512, heads=8, kv_heads=2, head_dim=64, inter=256, experts=8, top_k=2, vocab=2048, seed=4)
    chains = [example.TokenStep(3, 64, **kw) for _ in range(2)]
    chains[1].sampler.settings["top_p"][1] = float("nan")
    uniform = torch.rand((6, 3), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda")
    for t in range(6):
        for chain in chains:
            chain.step(uniform[t])
        torch.cuda.synchronize()
        good, bad = (chain.tokens.tolist() for chain in chains)
        assert bad == [good[0], -1, good[2]] and min(good) >= 0
        assert bool(torch.isfinite(chains[1].layer.out).all())
    assert int(chains[1].sampler.status.item()) == example.w4.W4A16_DEV_SETTING
    assert int(chains[0].sampler.status.item()) == 0
