"""w4a16_sample: the exactness of a token's share, temperatures down to the smallest, masked rows that end anywhere."""
import numpy as np
import pytest

from test_gpu_sample import ALL, Case, w4  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("top_k", [0, 2])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_logits_far_below_a_largest_near_zero(w4, dtype, top_k):  # noqa: F811
    """Two tokens, the first of share s = P / (1 + P): numbers just below s take it, numbers just above the other.

    P is held to 2^-30 of itself and half of 2^-43, which is 2^-30 of a P of 2^-14; s as well.  The numbers are
    s (1 -+ 2^-22.5), rounded by 2^-24 of themselves: further than 2^-23.6 from s.  The difference of logits, whose digits
    do not fit fp32, may not lose any: 2^-25 of it would be (t - l) / T 2^-25, up to 2^-22, of P.
    """
    import torch
    n = 4096
    rng = np.random.default_rng(5)
    to = lambda x: torch.from_numpy(x).to({"fp16": torch.float16, "bf16": torch.bfloat16}[dtype])
    top = to(np.exp2(rng.uniform(-13, -5, n)) * rng.choice([-1.0, 1.0], n))
    low = to(-np.exp2(rng.uniform(0, 12, n)))
    distance = (top.double() - low.double()).numpy()
    t = (distance / (rng.uniform(4, 14, n) * np.log(2))).astype(np.float32)
    p = np.exp(-distance / t.astype(np.float64))
    share = p / (1 + p)
    case = Case(1, dtype, 2 * n, 2, top_k=[top_k])
    case.logits.copy_(torch.stack((low, top), 1).repeat(2, 1))
    case.uniform.copy_(torch.from_numpy(np.concatenate((share * (1 - 2.0 ** -22.5), share * (1 + 2.0 ** -22.5)))).float())
    case.settings["temperature"] = torch.from_numpy(np.concatenate((t, t))).cuda()
    case.run(w4)
    torch.cuda.synchronize()
    got = case.tokens.cpu().numpy()
    assert int((got[:n] != 0).sum()) == 0 and int((got[n:] != 1).sum()) == 0, (int((got[:n] != 0).sum()), int((got[n:] != 1).sum()))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_the_smallest_temperatures(w4, dtype):  # noqa: F811
    """Temperatures below 2^-126 count as 2^-126, at which only bf16's subnormal numbers are near one another."""
    import torch
    heat = [2.0 ** -126, 2.0 ** -125, 2.0 ** -149, 1e-40, 2.0 ** -120]
    case = Case(2, dtype, 60, 300, temperature=heat, top_k=[0, 40], top_p=[1.0, 0.8, 0.9])
    bits = torch.randint(0, 100, (60, 300), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    case.logits[:] = bits.short().view(case.logits.dtype)  # subnormal numbers
    case.logits[::7, 5] = 1.0
    case.run(w4)
    torch.cuda.synchronize()
    case.settings["temperature"].clamp_(min=2.0 ** -126)
    case.check()
    assert int(case.status.item()) == 0


@pytest.mark.parametrize("vocab", [8 * 33, 8 * 31 + 3, 4096 + 8 * 5, 8 * 512 * 3 + 8 * 40 + 1, 50001, 131063])
@pytest.mark.parametrize("masked", [0.5, 0.9, 0.997])
def test_masked_rows_that_end_inside_a_warp(w4, vocab, masked):  # noqa: F811
    """Rows whose last turn takes part of a warp or of a block, from all masked but a few to half of them live."""
    case = Case(7, "fp16", 24, vocab, pad=3, masked=masked, **ALL)
    case.logits[:, vocab - 1] = 2.0
    case.logits[3, :vocab - 9] = float("-inf")
    case.run(w4)
    case.check()
    assert int(case.status.item()) == 0
