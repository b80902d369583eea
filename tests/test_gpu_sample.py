"""w4a16_sample against its definition in 64 bits.

Tolerance.  P is a multiple of 2^-43 good to 2^-30 of itself: a sum of P over a vocabulary of V is off by at most
V 2^-44 + 2^-30 sum, and a share of a sum by twice that.  So where a row's number falls further than
d = 2 (V 2^-44 + 2^-30 sum) from the borders that decide, the token is the definition's; where it does not, a token
next to the border is right too.  logprob: a share y / all of fp32 numbers is off by 3 roundings of 2^-24; its log, where
y <= all / 2, by that and by a unit of the result, where |log| >= 0.69: below 2^-21.5 |log|.  Above, of what is missing
from 1: log1p's condition is at most 1.45 there, so 4.4 2^-24 + 2^-23 of it, below 2^-21 |log|.  With the error of P
itself: |log - ref| <= 2^-21 |ref| + 2^-29 + V 2^-43 / P.
"""
import numpy as np
import pytest

import kv4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import weight_only_int4_03_gb300 as w4
    return w4


def kept_tokens(w, order, k, p, least):
    if k > 0:
        order = order[:k]
    if p < 1:
        sums = np.cumsum(w[order])
        want = max(p, 0.0) * sums[-1]
        order = order[:max(1, int((sums - w[order] < want).sum()))]
    return np.sort(order[(w[order] >= min(least, 1.0)) & (w[order] > 0)])


def answers(x, u, t, k, p, least):
    """{token: logprob} of the tokens that are right for a row of logits in 64 bits."""
    x = np.where(np.isnan(x), -np.inf, x)
    if x.max() == -np.inf:
        return {-1: -np.inf}
    if t == 0:
        return {int(np.argmax(x)): 0.0}
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(x == x.max(), 1.0, np.exp((x - x.max()) / t))
    order = np.argsort(-x, kind="stable")
    total = w.sum()
    d = 2 * (x.size * 2.0 ** -44 + 2.0 ** -30 * total)
    found = {}
    for e in ((0.0,) if not p < 1 else (0.0, -d / total, d / total)):
        kept = kept_tokens(w, order, k, p + e, least)
        sums = np.cumsum(w[kept])
        for target in (u * sums[-1] - d, u * sums[-1], u * sums[-1] + d):
            at = min(int(np.searchsorted(sums, max(target, 0.0), side="right")), kept.size - 1)
            found.setdefault(int(kept[at]), float(np.log(w[kept[at]] / sums[-1])))
    return found


class Case:
    def __init__(self, seed, dtype, batch, vocab, sigma=3.0, pad=0, shift=0, masked=0.0, **settings):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = kv4.TYPES[dtype]
        self.dtype, self.batch, self.vocab, self.ld = dtype, batch, vocab, vocab + pad
        x = torch.randn(batch * self.ld + shift, generator=g, device="cuda") * sigma
        if masked:
            x[torch.rand(x.shape, generator=g, device="cuda") < masked] = float("-inf")
        self.logits = x.to(dt)[shift:].view(batch, self.ld)
        self.logits[:, vocab:] = 1000.0  # must not be looked at
        self.uniform = torch.rand(batch, generator=g, device="cuda")
        self.settings = {}
        for name, values in settings.items():
            kind = torch.int32 if name == "top_k" else torch.float32
            self.settings[name] = torch.tensor([values[i % len(values)] for i in range(batch)], dtype=kind, device="cuda")
        self.tokens = torch.full((batch,), -7, dtype=torch.int32, device="cuda")
        self.logprobs = torch.full((batch,), 7.0, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, w4, **kw):
        w4.w4a16_sample(self.logits, self.uniform, self.tokens, self.batch, self.vocab,
                        w4.W4A16_FLAG_BF16 if self.dtype == "bf16" else 0, logprobs=self.logprobs, status=self.status,
                        ld=self.ld, **self.settings, **kw)

    def column(self, name, default):
        v = self.settings.get(name)
        return [default] * self.batch if v is None else v.tolist()

    def check(self, rows=None):
        import torch
        torch.cuda.synchronize()
        x = self.logits[:, :self.vocab].double().cpu().numpy()
        got, logs = self.tokens.tolist(), self.logprobs.tolist()
        each = list(zip(self.uniform.tolist(), self.column("temperature", 1.0), self.column("top_k", 0),
                        self.column("top_p", 1.0), self.column("min_p", 0.0)))
        for i in range(self.batch) if rows is None else rows:
            right = answers(x[i], *each[i])
            assert got[i] in right, (i, got[i], right, each[i])
            ref = right[got[i]]
            if ref == -np.inf:
                assert logs[i] == -np.inf
            else:
                tol = 2.0 ** -21 * abs(ref) + 2.0 ** -29 + self.vocab * 2.0 ** -43 * np.exp(-ref)
                assert abs(logs[i] - ref) <= tol, (i, logs[i], ref)


OPEN = dict()
TOP_K = dict(top_k=[1, 2, 7, 50, 1000, 0, -3, 10 ** 6])
TOP_P = dict(top_p=[0.9, 0.0, 0.5, 1e-6, 0.999999, 1.0, 2.0, -1.0])
MIN_P = dict(min_p=[0.0, 0.05, 0.5, 1.0, 3.0, -1.0, 1e-9])
HEAT = dict(temperature=[1.0, 0.0, 0.3, 2.5, 0.05, 100.0, 1e-20, 1e30])
ALL = dict(temperature=[1.0, 0.7, 1.3, 0.0, 0.5], top_k=[0, 40, 1000, 3], top_p=[0.95, 1.0, 0.7], min_p=[0.0, 0.02])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kw", [
    dict(batch=1, vocab=1), dict(batch=3, vocab=7, **TOP_K), dict(batch=9, vocab=100, **TOP_P),
    dict(batch=16, vocab=1000, **TOP_K), dict(batch=16, vocab=2049, pad=7, **TOP_P),
    dict(batch=1, vocab=32000, **dict(top_k=[40], top_p=[0.95], temperature=[0.7])),
    dict(batch=16, vocab=32001, pad=5, shift=1, **HEAT), dict(batch=7, vocab=65537, pad=255, **MIN_P),
    dict(batch=60, vocab=50003, pad=5, **ALL), dict(batch=60, vocab=50003, pad=5, masked=0.999, **ALL),
    dict(batch=60, vocab=20000, sigma=0.0, **ALL), dict(batch=60, vocab=20000, sigma=0.01, **ALL),
    dict(batch=60, vocab=20000, sigma=40.0, **ALL), dict(batch=400, vocab=3001, pad=7, **ALL),
    dict(batch=3, vocab=524288, **dict(top_p=[1.0, 0.9, 0.99], top_k=[0, 0, 100000])), dict(batch=40, vocab=131071, pad=1),
], ids=lambda c: f"b{c['batch']}v{c['vocab']}" + "".join(c.keys() - {"batch", "vocab"}))
def test_matches_definition(w4, kw, dtype):
    case = Case(3, dtype, **kw)
    case.run(w4)
    case.check()
    assert int(case.status.item()) == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_ends_of_the_uniform_numbers(w4, dtype):
    import torch
    case = Case(4, dtype, 12, 9001, pad=7, **ALL)
    case.uniform.fill_(0.0)
    case.run(w4)
    case.check()
    case.uniform.fill_(1.0 - 2.0 ** -24)
    case.run(w4)
    case.check()
    assert int(case.status.item()) == 0


def test_equal_logits_go_by_index(w4):
    """Ties at the thresholds: the lowest indices are kept, whichever block or warp has them."""
    import torch
    case = Case(5, "fp16", 8, 40000, sigma=0.0, top_k=[5], temperature=[1.0])
    at = torch.randperm(40000, generator=torch.Generator().manual_seed(1))[:300].sort().values.cuda()
    case.logits.fill_(-2.0)
    case.logits[:, at] = 3.0  # 300 of them are the largest
    case.logits[4:, at[::2]] = 4.0  # in these rows every other one is larger
    case.settings["top_k"] = torch.tensor([5, 300, 299, 1, 5, 150, 151, 450], dtype=torch.int32, device="cuda")
    for u in (0.0, 0.19, 0.21, 0.5, 0.81, 0.999, 1.0 - 2.0 ** -24):
        case.uniform.fill_(u)
        case.run(w4)
        case.check()
    case.uniform.fill_(1.0 - 2.0 ** -24)
    case.run(w4)
    torch.cuda.synchronize()
    assert case.tokens[:4].tolist() == [int(at[4]), int(at[299]), int(at[298]), int(at[0])]
    assert case.tokens[4:6].tolist() == [int(at[8]), int(at[298])]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_infinities_nan_zeros_and_rows_of_nothing(w4, dtype):
    import torch
    case = Case(6, dtype, 16, 5000, temperature=[1.0, 1.0, 0.0], top_k=[0, 40], top_p=[1.0, 0.9])
    x = case.logits
    x[0] = float("-inf")
    x[1] = float("nan")
    x[2] = float("-inf")
    x[3, 1:] = float("-inf")
    x[4, ::3] = float("nan")
    x[5, 7], x[5, 4000], x[5, 4001] = float("inf"), float("inf"), float("nan")
    x[6] = 0.0
    x[6, ::2] = -0.0
    x[7] = -0.0
    x[8] = torch.finfo(x.dtype).max
    x[9] = torch.finfo(x.dtype).min
    x[10] = torch.finfo(x.dtype).min
    x[10, 17] = torch.finfo(x.dtype).max
    x[11] = torch.finfo(x.dtype).tiny
    x[12, :4999] = float("-inf")
    case.run(w4)
    case.check()
    assert case.tokens[:3].tolist() == [-1, -1, -1] and case.tokens[12] == 4999
    assert int(case.status.item()) == 0
    # Rows whose largest logits are infinite, with each kind of setting.
    case = Case(9, dtype, 24, 5000, temperature=[1.0], top_k=[0, 1, 2, 40, 200, 3000], top_p=[1.0, 1.0, 1.0, 0.5])
    for i in range(24):
        case.logits[i, 11 + i:11 + 200 * (1 + i % 7):3] = float("inf")
    case.run(w4)
    case.check()
    assert int(case.status.item()) == 0


def test_settings_out_of_range_are_reported(w4):
    import torch
    nan, inf = float("nan"), float("inf")
    case = Case(7, "fp16", 9, 1000, temperature=[1.0], top_k=[3], top_p=[0.5], min_p=[0.1])
    case.settings["temperature"][:3] = torch.tensor([nan, -1.0, inf])
    case.settings["top_p"][3] = nan
    case.settings["min_p"][4] = nan
    case.uniform[5:8] = torch.tensor([1.0, -0.5, nan])
    case.run(w4)
    torch.cuda.synchronize()
    assert case.tokens[:8].tolist() == [-1] * 8 and bool(torch.isnan(case.logprobs[:8]).all())
    assert int(case.status.item()) == w4.W4A16_DEV_SETTING
    case.check(rows=[8])
    case.settings["temperature"].fill_(0.0)  # takes the largest whatever the uniform number
    case.settings["top_p"].fill_(1.0)
    case.settings["min_p"].fill_(0.0)
    case.status.zero_()
    case.run(w4)
    case.check()
    assert int(case.status.item()) == 0


def test_many_rows_of_few_tokens(w4):
    case = Case(10, "fp16", 70001, 9, pad=2, shift=3, **ALL)
    case.run(w4)
    case.check(rows=range(0, 70001, 101))
    assert int(case.status.item()) == 0 and bool((case.tokens >= 0).all())


def test_repeats_batches_and_graphs_agree(w4):
    """A row's token does not depend on the other rows, the stream or the number of blocks that hold it."""
    import torch
    case = Case(8, "bf16", 300, 30011, pad=5, **ALL)
    case.run(w4)
    case.check()
    want, logs = case.tokens.clone(), case.logprobs.clone()
    for i in (0, 1, 17, 299):
        one = {n: v[i:i + 1] for n, v in case.settings.items()}
        token, log = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda")
        w4.w4a16_sample(case.logits[i], case.uniform[i:], token, 1, case.vocab, w4.W4A16_FLAG_BF16, logprobs=log, **one)
        torch.cuda.synchronize()
        assert int(token) == int(want[i]) and float(log) == float(logs[i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            case.run(w4, stream=side)
        case.tokens.fill_(-9)
        graph.replay()
        graph.replay()
    side.synchronize()
    assert torch.equal(case.tokens, want) and torch.equal(case.logprobs, logs)


def test_shares_are_those_of_the_exponential(w4):
    """logprob of every token of a row, one after the other, against the 64-bit softmax."""
    import torch
    n = 3001
    logits = (torch.randn(n, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") * 6).half()
    w = torch.softmax(logits.double() / 0.9, 0)
    middle = ((w.cumsum(0) - w / 2)).float().clamp(max=1 - 2.0 ** -24)
    tokens, logs = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, device="cuda")
    w4.w4a16_sample(logits.expand(n, n).contiguous(), middle, tokens, n, n,
                    temperature=torch.full((n,), 0.9, device="cuda"), logprobs=logs)
    torch.cuda.synchronize()
    wide = w > 2.0 ** -20  # the uniform numbers' steps of 2^-24 do not reach the others' middles
    assert torch.equal(tokens[wide].long(), torch.arange(n, device="cuda")[wide])
    ref = torch.log(w[tokens.long()])
    # 0.9 is rounded to fp32: 2^-25 of the logits' distance, at most 60.  P is rounded to a multiple of 2^-43, which is
    # off by half of one: of a P, the largest being 1, by up to 2^-44 / P of itself, and -log(1 - x) <= 1.1 x for x <= 0.1.
    half = 1.1 * 2.0 ** -44 * w.max() / w[tokens.long()]
    assert float(half.max()) < 0.1
    assert bool(((logs.double() - ref).abs() <= 2.0 ** -21 * ref.abs() + 2.0 ** -29 + 2 * 60 * 2.0 ** -25 + half).all())
