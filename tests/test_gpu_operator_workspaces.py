"""One workspace, zero-filled once, under calls of sizes that come and go as in a server whose batch
changes: every call gives the bits that it gives in a zeroed workspace of its own, and those are the
operator's (the tolerances are those of the operators' own tests)."""
import pytest

from test_gpu_attention import Case
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


def test_attention_at_changing_batches_and_widths(w4):
    """Partial results of one call never lie where another call counts arrivals: single long sequences
    between batches of thousands of rows, three head widths."""
    import torch
    cases = dict(
        long=Case(41, "bf16", [9001], 40, 8, 128, 32),
        wide=Case(42, "fp16", [37 * i % 700 for i in range(300)], 16, 8, 128, 16),
        d256=Case(43, "fp16", [5000, 17], 8, 2, 256, 16),
        many=Case(44, "bf16", [53 * i % 300 for i in range(1500)], 8, 4, 64, 16),
        one=Case(45, "fp16", [20000], 8, 1, 64, 64),
        two=Case(46, "bf16", [20000, 9], 8, 1, 256, 64, window=15000),
    )
    alone = {}
    for name, case in cases.items():
        case.run(w4, case.workspace(w4))
        case.check()
        alone[name] = case.out.clone(), case.lse.clone()
    shared = max((case.workspace(w4) for case in cases.values()), key=lambda ws: ws.numel())
    for name in ("long", "wide", "d256", "many", "long", "one", "many", "two", "wide", "d256", "many", "one", "wide"):
        case = cases[name]
        for x in (case.out, case.lse):
            x.fill_(float("nan"))
        case.run(w4, shared)
        torch.cuda.synchronize()
        assert torch.equal(case.out, alone[name][0]) and torch.equal(case.lse, alone[name][1]), name
    assert w4.w4a16_status(shared) == 0


@pytest.mark.parametrize("n,k", [(28672, 4096), (4096, 4096), (12288, 1024), (4096, 14336)])
def test_gemm_at_changing_row_counts(w4, n, k):
    """The products around the operators, from a single token to prompts and back, dense and grouped."""
    import torch
    flags, wt = w4.W4A16_FLAG_IS_K_FULL, w4.W4A16_TYPE_U4B8
    g = torch.Generator(device="cuda").manual_seed(47)
    words = torch.randint(-2 ** 31, 2 ** 31 - 1, (k // 8, n), generator=g, device="cuda", dtype=torch.int32)
    scales = torch.rand((k // 128, n), generator=g, device="cuda").mul_(0.02).half()
    packed = torch.empty(k * n // 8, dtype=torch.int32, device="cuda")
    w4.w4_repack(words, None, packed, k, n)
    # Two experts with the same weights: every token once, split unevenly.
    packed2, scales2 = packed.repeat(2), scales.repeat(2, 1, 1)
    zeroed = lambda size: torch.zeros(size, dtype=torch.uint8, device="cuda")

    def dense(m, x, out, ws):
        w4.w4a16_gemm(x, packed, out, scales, None, None, None, ws, m, n, k, 128, wt, flags)

    def grouped(m, x, out, ws):
        off = torch.tensor([0, m // 3, m], dtype=torch.int32, device="cuda")
        ids, rows = (torch.arange(c, dtype=torch.int32, device="cuda") for c in (2, m))
        w4.w4a16_gemm_grouped(x, packed2, out, scales2, None, ids, off, rows, rows, 2, 2, m, m, n, k, 128, wt, flags, ws)

    calls = {dense: lambda m: w4.w4a16_workspace_size(m, n, k, 128, flags),
             grouped: lambda m: w4.w4a16_grouped_workspace_size(m, 2, n, k, 128, flags)}
    counts = (1, 16, 512, 33, 1000, 4096, 64, 2000, 7)
    shared = zeroed(max(size(m) for size in calls.values() for m in counts))
    for m in counts:
        x = torch.randn((m, k), generator=g, device="cuda", dtype=torch.float16)
        for call, size in calls.items():
            alone, out = (torch.full((m, n), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2))
            call(m, x, alone, zeroed(size(m)))
            call(m, x, out, shared)
            torch.cuda.synchronize()
            assert bool(torch.isfinite(alone).all())
            assert torch.equal(out, alone), (call.__name__, m)
    assert w4.w4a16_status(shared) == 0
