"""w4a16_moe_layer against its definition in 64 bits.

Tolerance.  Every operand of the products is exact; a 64-row block's sum is an fp32 sum of eight MMA
steps whose partial sums stay below 15 (fp16; 143 with bf16's offset of 128) times |sum a|'s size, so a
column's relative error is below 2^-14 (bf16: 2^-12) of its own root mean square, and the remainder
kept beside h adds 2^-17 at most.  act and the product of gate and up multiply relative errors by
less than 3.  With u = 2^-11 / 2^-8 for the last rounding:
    |y - ref| <= u |ref| + 2^-12 r  (fp16),   u |ref| + 2^-10 r  (bf16),
r the root mean square of the token's expert sum.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

UNIT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}
REL = {"fp16": 2.0 ** -12, "bf16": 2.0 ** -10}


@pytest.fixture(scope="module")
def w4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import weight_only_int4_03_gb300 as w4
    return w4


def unpack(words):
    """[K/8, N] words -> [K, N] codes, low nibble first."""
    import torch
    return torch.stack([(words >> (4 * i)) & 15 for i in range(8)], 1).flatten(0, 1)


class Layer:
    def __init__(self, w4, seed, dtype, tokens, hidden, inter, experts, top, group_size=128, zeros=False,
                 act="silu", renorm=True, residual=True, pad=0, router_sigma=2.0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = torch.float16 if dtype == "fp16" else torch.bfloat16
        self.__dict__.update(w4=w4, dtype=dtype, tokens=tokens, hidden=hidden, inter=inter, experts=experts,
                             top=top, group_size=group_size, act=act, renorm=renorm, pad=pad)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=dt)
        self.x = rnd(tokens, hidden + pad)
        self.router = rnd(experts, hidden) * (router_sigma / math.sqrt(hidden))
        self.residual = rnd(tokens, hidden + pad) if residual else None
        self.weights = []
        for k, n in ((hidden, 2 * inter), (inter, hidden)):
            groups = 1 if group_size == -1 else k // group_size
            words = torch.randint(-2 ** 31, 2 ** 31 - 1, (experts, k // 8, n), generator=g, device="cuda",
                                  dtype=torch.int32)
            s = (torch.rand((experts, groups, n), generator=g, device="cuda") * 0.019 + 0.001).to(dt)
            z = torch.randint(0, 16, (experts, groups, n), generator=g, device="cuda").to(dt) if zeros else None
            self.weights.append((words, s, z))
        self.flags = (w4.W4A16_FLAG_SWIGLU if act == "silu" else w4.W4A16_FLAG_GEGLU) | (
            w4.W4A16_FLAG_BF16 if dtype == "bf16" else 0) | (w4.W4A16_FLAG_HAS_ZP if zeros else 0) | (
            w4.W4A16_FLAG_MOE_RENORM if renorm else 0)
        self.weight_type = w4.W4A16_TYPE_U4 if zeros else w4.W4A16_TYPE_U4B8

        def interleave(a):
            if a is None:
                return None
            out = torch.empty_like(a)
            w4.w4_gate_up_interleave(a, out, a.shape[0] * a.shape[1], 2 * inter)
            return out

        def pack(words, k, n):
            out = torch.empty((experts, k * n // 8), dtype=torch.int32, device="cuda")
            for e in range(experts):
                w4.w4_repack(words[e], None, out[e], k, n)
            return out

        (uw, us, uz), (dw, ds, dz) = self.weights
        self.packed = (pack(interleave(uw), hidden, 2 * inter), interleave(us), interleave(uz),
                       pack(dw, inter, hidden), ds, dz)
        self.ws = torch.zeros(w4.w4a16_moe_layer_workspace_size(tokens, hidden, inter, experts, top),
                              dtype=torch.uint8, device="cuda")
        self.y = torch.full((tokens, hidden + pad), float("nan"), dtype=dt, device="cuda")
        self.ids = torch.full((tokens, top), -1, dtype=torch.int32, device="cuda")
        self.tw = torch.full((tokens, top), float("nan"), device="cuda")
        torch.cuda.synchronize()

    def run(self, y=None, **kw):
        ld = self.hidden + self.pad
        self.w4.w4a16_moe_layer(self.x, self.router, *self.packed, self.y if y is None else y, self.ws,
                                self.tokens, self.hidden, self.inter, self.experts, self.top, self.group_size,
                                self.weight_type, self.flags, residual=self.residual, topk_ids=self.ids,
                                topk_weights=self.tw, ldx=ld, ldy=ld, ldr=ld, **kw)

    def matrix(self, which, e):
        import torch
        words, s, z = self.weights[which]
        q = unpack(words[e]).double()
        groups = s.shape[1]
        rep = lambda a: a[e].double().repeat_interleave(q.shape[0] // groups, 0)
        return (q - (8.0 if z is None else rep(z))) * rep(s)

    def reference(self):
        """(expert sums [t, hidden], ids, weights) in fp64."""
        import torch
        x = self.x[:, :self.hidden].double()
        logits = x @ self.router.double().t()
        p = torch.softmax(logits, 1)
        order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :self.top]
        w = p.gather(1, order)
        if self.renorm:
            w = w / w.sum(1, keepdim=True)
        y = torch.zeros_like(x)
        for e in sorted(set(order.flatten().tolist())):
            tok, slot = torch.nonzero(order == e, as_tuple=True)
            gu = x[tok] @ self.matrix(0, e)
            gate, up = gu[:, :self.inter], gu[:, self.inter:]
            if self.act == "silu":
                h = gate * torch.sigmoid(gate) * up
            else:
                h = 0.5 * gate * (1 + torch.tanh(math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3))) * up
            y.index_add_(0, tok, w[tok, slot][:, None] * (h @ self.matrix(1, e)))
        return y, order, w

    def check(self, y=None):
        import torch
        torch.cuda.synchronize()
        s, ids, w = self.reference()
        assert torch.equal(self.ids.long(), ids)
        assert bool(((self.tw.double() - w).abs() <= 2.0 ** -18 * w + 1e-30).all())
        ref = s + (self.residual[:, :self.hidden].double() if self.residual is not None else 0.0)
        got = (self.y if y is None else y)[:, :self.hidden].double()
        r = s.pow(2).mean(1, keepdim=True).sqrt()
        err = (got - ref).abs()
        tol = UNIT[self.dtype] * ref.abs() + REL[self.dtype] * r
        assert bool((err <= tol).all()), f"{float((err / tol).max())} times the tolerance"
        assert self.w4.w4a16_status(self.ws) == 0


CASES = [
    dict(dtype="fp16", tokens=1, hidden=256, inter=128, experts=1, top=1),
    dict(dtype="bf16", tokens=1, hidden=256, inter=128, experts=4, top=2, group_size=64),
    dict(dtype="fp16", tokens=1, hidden=1024, inter=1792, experts=8, top=2),
    dict(dtype="bf16", tokens=3, hidden=512, inter=384, experts=60, top=4, act="gelu"),
    dict(dtype="fp16", tokens=5, hidden=768, inter=256, experts=9, top=3, zeros=True, renorm=False),
    dict(dtype="bf16", tokens=8, hidden=512, inter=640, experts=4, top=4, zeros=True, group_size=64),
    dict(dtype="fp16", tokens=9, hidden=512, inter=512, experts=16, top=1, group_size=256),
    dict(dtype="fp16", tokens=17, hidden=512, inter=256, experts=2, top=1, group_size=-1),
    dict(dtype="bf16", tokens=33, hidden=256, inter=256, experts=3, top=2, residual=False),
    dict(dtype="fp16", tokens=64, hidden=512, inter=384, experts=2, top=2, act="gelu"),   # 64 pairs an expert
    dict(dtype="bf16", tokens=64, hidden=256, inter=128, experts=1, top=1, group_size=64),
    dict(dtype="fp16", tokens=64, hidden=512, inter=256, experts=128, top=8, pad=8),
    dict(dtype="bf16", tokens=40, hidden=256, inter=128, experts=512, top=16, router_sigma=1.0),
    dict(dtype="fp16", tokens=2, hidden=2048, inter=768, experts=128, top=8),
    dict(dtype="fp16", tokens=6, hidden=1792, inter=2816, experts=5, top=2, zeros=True),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_matches_definition(w4, kw):
    layer = Layer(w4, 21, **kw)
    layer.run()
    layer.check()


def test_repeats_are_bit_identical_in_place_and_in_a_graph(w4):
    import torch
    layer = Layer(w4, 22, "bf16", 20, 512, 768, 16, 4, zeros=True)
    layer.run()
    torch.cuda.synchronize()
    first = layer.y.clone()
    layer.check()
    for _ in range(5):
        layer.run()
    torch.cuda.synchronize()
    assert torch.equal(layer.y, first)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            layer.run(stream=side)
        layer.y.fill_(float("nan"))
        graph.replay()
    side.synchronize()
    assert torch.equal(layer.y, first)
    keep = layer.residual.clone()
    layer.run(y=layer.residual)  # the residual stream updated where it lies
    torch.cuda.synchronize()
    assert torch.equal(layer.residual, first)
    layer.residual.copy_(keep)


def test_equal_scores_choose_the_lowest_experts(w4):
    """A router of equal rows: every score ties, the lowest indices win, in order."""
    layer = Layer(w4, 23, "fp16", 3, 256, 128, 40, 5)
    layer.router[:] = layer.router[0]
    layer.run()
    layer.check()
    assert layer.ids.tolist() == [[0, 1, 2, 3, 4]] * 3


def test_a_bad_token_leaves_the_others_alone(w4):
    """NaN in one token's row: its output is NaN, its experts are distinct and in range, and every
    other token's bits are as without it."""
    import torch
    layer = Layer(w4, 24, "fp16", 6, 256, 128, 8, 2)
    layer.run()
    torch.cuda.synchronize()
    clean = layer.y.clone()
    layer.x[2] = float("nan")
    layer.run()
    torch.cuda.synchronize()
    assert bool(torch.isnan(layer.y[2]).all())
    ids = layer.ids[2].tolist()
    assert len(set(ids)) == 2 and all(0 <= e < 8 for e in ids)
    other = [0, 1, 3, 4, 5]
    assert torch.equal(layer.y[other], clean[other])


def test_large_inner_activations_stay_finite_in_fp16(w4):
    """h beyond fp16's range: its value part stops at 65504 and the remainder carries the rest."""
    import torch
    layer = Layer(w4, 25, "fp16", 2, 256, 128, 1, 1, residual=False)
    (uw, us, uz), (dw, ds, dz) = layer.weights
    ds *= 2.0 ** -6
    base = layer.x.double()

    def h_of(x):
        gu = x @ layer.matrix(0, 0)
        return gu[:, :128] * torch.sigmoid(gu[:, :128]) * gu[:, 128:]

    c = 1.0
    for _ in range(8):  # x such that the largest |h| is near 1e5
        layer.x.copy_((base * c).half())
        c *= math.sqrt(1e5 / float(h_of(layer.x.double()).abs().max()))
    assert 65504 < float(h_of(layer.x.double()).abs().max()) < 131008
    layer.run()
    assert bool(torch.isfinite(layer.y).all())
    layer.check()


@pytest.mark.parametrize("dtype,tokens,experts,top", [
    ("fp16", 8, 8, 4), ("bf16", 2, 512, 16), ("fp16", 1, 16, 16),   # up to 32 pairs: grouped by one warp
    ("fp16", 11, 3, 3), ("bf16", 8, 60, 5), ("fp16", 9, 16, 4),     # more; one level of routing, and two
    ("bf16", 64, 512, 16), ("fp16", 64, 16, 16),                    # the largest tables; every expert 64 pairs
])
def test_routing_sizes(w4, dtype, tokens, experts, top):
    layer = Layer(w4, 26, dtype, tokens, 256, 128, experts, top, group_size=64, router_sigma=1.0)
    for _ in range(2):
        layer.y.fill_(float("nan"))
        layer.run()
        layer.check()


@pytest.mark.parametrize("dtype,tokens,experts,top", [("fp16", 1, 8, 2), ("bf16", 6, 16, 4), ("fp16", 20, 4, 2)])
def test_new_inputs_in_one_workspace(w4, dtype, tokens, experts, top):
    """Nothing of a call is left in the next: the same layer on other rows, back to back."""
    import torch
    layer = Layer(w4, 27, dtype, tokens, 512, 384, experts, top, zeros=True)
    rows = [torch.randn_like(layer.x) * s for s in (1.0, 0.5, 2.0, 1.0)]
    outs = [torch.empty_like(layer.y) for _ in rows]
    for x, y in zip(rows, outs):
        layer.x.copy_(x)
        layer.run(y=y)
    for x, y in zip(rows, outs):
        layer.x.copy_(x)
        layer.ws.zero_()
        layer.run()
        torch.cuda.synchronize()
        assert torch.equal(layer.y, y)
        layer.check()


@pytest.mark.parametrize("most", [2e5, 1e7])
@pytest.mark.parametrize("kw", [
    dict(tokens=1, hidden=256, inter=384, experts=1, top=1),
    dict(tokens=4, hidden=512, inter=256, experts=8, top=2, group_size=64, act="gelu"),
    dict(tokens=20, hidden=256, inter=512, experts=4, top=2, zeros=True),
    dict(tokens=64, hidden=256, inter=256, experts=3, top=2, group_size=-1, renorm=False, pad=8),
], ids=lambda c: f"t{c['tokens']}e{c['experts']}" if isinstance(c, dict) else f"{c:g}")
def test_inner_activations_of_any_size_in_fp16(w4, kw, most):
    """h far beyond both of its 16-bit parts in every third token, beside tokens of ordinary size: the
    outputs are finite and within the tolerance of every other call, and calls repeat their bits."""
    import torch
    layer = Layer(w4, 28, "fp16", residual=False, router_sigma=1e-3, **kw)
    layer.weights[1][1].mul_(2.0 ** -9)  # the down scales: outputs inside fp16's range
    rows = torch.arange(layer.tokens, device="cuda") % 3 == 0
    base = layer.x[rows].double()

    def h_of(x):
        gu = x[:, :layer.hidden].double() @ layer.matrix(0, 0)
        gate, up = gu[:, :layer.inter], gu[:, layer.inter:]
        return (gate * torch.sigmoid(gate) * up).abs().max()

    c = 1.0
    for _ in range(8):
        layer.x[rows] = (base * c).half()
        c *= math.sqrt(most / float(h_of(layer.x[rows])))
    assert float(h_of(layer.x[rows])) > 0.9 * most > 131008
    layer.run()
    assert bool(torch.isfinite(layer.y[:, :layer.hidden]).all())
    layer.check()
    first = layer.y.clone()
    for _ in range(3):
        layer.run()
    torch.cuda.synchronize()
    assert torch.equal(layer.y[:, :layer.hidden], first[:, :layer.hidden])
    # Nothing of it is left in the next call.
    layer.x[rows] = base.half()
    layer.run()
    layer.check()


@pytest.mark.parametrize("dtype,tokens,hidden,inter,experts,favoured", [
    ("fp16", 64, 512, 16384, 32, (3, 30)),   # 64 pairs on each of two experts where four are expected; drawn units
    ("bf16", 64, 512, 1024, 128, (0, 127)),
    ("fp16", 33, 256, 2048, 128, (64,)),     # one expert for every token
    ("bf16", 9, 1024, 512, 60, (7, 8, 9)),
])
def test_skewed_routing(w4, dtype, tokens, hidden, inter, experts, favoured):
    """Every token chooses the same few experts: many times the pairs of an even spread on each."""
    import torch
    layer = Layer(w4, 29, dtype, tokens, hidden, inter, experts, len(favoured), group_size=64, router_sigma=0.5)
    g = torch.Generator(device="cuda").manual_seed(30)
    common = torch.randn(hidden, generator=g, device="cuda")
    layer.x += common.to(layer.x.dtype)
    for i, e in enumerate(favoured):
        layer.router[e] = ((6 + 0.25 * i) * common / hidden).to(layer.router.dtype)
    for _ in range(2):
        layer.y.fill_(float("nan"))
        layer.run()
        layer.check()
    assert sorted(set(layer.ids.flatten().tolist())) == sorted(favoured)
