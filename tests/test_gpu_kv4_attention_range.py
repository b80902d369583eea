"""w4a16_kv4_attention where precision and range could run out: weights in bf16, large steps, queries of a wide range.

Tolerance, as beside the operator's other tests but for p s, which goes on with 2^-22 of itself in both types:
|out - ref| <= u |ref| + (4 E + 2^-17) R and |lse - ref| <= E + 2^-20 + 2^-22 |ref|, with R the largest of |value| and
16 |s|, u half a step of the type and E what a score is off by: (D / 16 + 6) 2^-23 B, B = scale max_i sum |q| (|s| c + |b|),
and what queries lose on their way to fp16.  The largest of a head is scaled to [2^13, 2^14), every second value to a
sixteenth of that; half a unit of the smallest fp16 numbers, 2^-25, is then at most 2^-25 16 / 2^13 = 2^-34 of the largest
query, and meets codes times steps: 2^-34 scale max |q| max_i sum |s| c.
"""
import pytest

import kv4
from test_gpu_kv4_attention import Case, w4  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def check(case):
    import torch
    torch.cuda.synchronize()
    group = case.heads // case.kv
    codes, params = (x.flatten(1, 2) for x in kv4.read(case.cache, case.page, case.kv, case.dim, case.group_size, case.dtype))
    for i, n in enumerate(case.lens_list):
        at = case.slots[i]
        sides = [kv4.values(codes[s][at], params[s][at]) for s in range(2)]
        got = case.out[i].view(case.heads, case.dim).double()
        q = case.q[i].view(case.kv, group, case.dim).double()
        logits = torch.einsum("cgd,ncd->cgn", q, sides[0]) * case.scale
        ref = torch.einsum("cgn,ncd->cgd", torch.softmax(logits, -1), sides[1]).reshape(case.heads, case.dim)
        lse = torch.logsumexp(logits, -1).reshape(case.heads)
        s, b = (params[0][at][..., j].double() for j in range(2))
        steps = codes[0][at].unflatten(-1, (s.shape[-1], -1)) * s.abs().unsqueeze(-1)
        weight = (steps + b.abs().unsqueeze(-1)).flatten(-2)
        bound = float((torch.einsum("cgd,ncd->cgn", q.abs(), weight) * case.scale).max())
        lost = 2.0 ** -34 * case.scale * float(q.abs().max()) * float(steps.flatten(-2).sum(-1).max())
        e = (case.dim / 16 + 6) * 2.0 ** -23 * bound + lost
        r = max(float(sides[1].abs().max()), 16 * float(params[1][at][..., 0].double().abs().max()))
        tol = kv4.UNIT[case.dtype] * ref.abs() + (4 * e + 2.0 ** -17) * r + 2.0 ** -25
        err = (got - ref).abs()
        assert bool((err <= tol).all()), f"sequence {i} (length {n}): {float((err / tol).max())} times the tolerance"
        off = (case.lse[i].double() - lse).abs()
        assert bool((off <= e + 2.0 ** -20 + 2.0 ** -22 * lse.abs()).all()), (i, float(off.max()), e)


@pytest.mark.parametrize("heads,kv,dim,group_size", [(8, 2, 128, -1), (10, 2, 128, 64), (6, 6, 64, -1), (12, 1, 64, -1),
                                                     (16, 1, 128, 64), (8, 1, 256, -1), (6, 2, 256, 128), (4, 1, 256, 64)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_values_that_nearly_cancel(w4, dtype, heads, kv, dim, group_size):  # noqa: F811
    """A few positions of nearly equal weights: outputs near zero show what each weight was rounded to."""
    case = Case(w4, 31, dtype, [2 + i % 9 for i in range(40)] + [700], heads, kv, dim, 16, group_size, q_sigma=2.0 ** -4)
    ws = case.workspace()
    case.run(ws)
    check(case)
    assert w4.w4a16_status(ws) == 0


@pytest.mark.parametrize("sigma", [2.0 ** 112, 2.0 ** 117, 2.0 ** 119, 2.0 ** -112])
@pytest.mark.parametrize("dim,group_size", [(64, -1), (128, 64), (256, -1)])
def test_values_of_the_types_whole_range(w4, dim, group_size, sigma):  # noqa: F811
    """Values in bf16 up to 2^122: steps up to 2^119."""
    import torch
    case = Case(w4, 32, "bf16", [1, 3, 17, 33], 4, 2, dim, 16, group_size)
    every = torch.cat(case.slots)
    g = torch.Generator(device="cuda").manual_seed(33)
    k, v = (torch.randn((every.numel(), 2, dim), generator=g, device="cuda", dtype=torch.float64).clamp(-4, 4)
            for _ in range(2))
    w4.w4a16_kv4_append(None, k.bfloat16(), (v * sigma).bfloat16(), None, None, 0.0, None, case.cache, None, None, every, None,
                        every.numel(), 0, 2, dim, 0, (), 0, 16, case.n_pages, group_size, case.flags)
    ws = case.workspace()
    case.run(ws)
    check(case)
    assert w4.w4a16_status(ws) == 0


@pytest.mark.parametrize("dtype,low", [("fp16", -14), ("bf16", -40)])
def test_queries_of_a_wide_range(w4, dtype, low):  # noqa: F811
    """Sizes from 2^low to 1 inside a head (and heads of different sizes), the largest at even and at odd places."""
    import torch
    case = Case(w4, 34, dtype, [5, 200], 16, 2, 128, 16, 64, sigma=64.0)
    g = torch.Generator(device="cuda").manual_seed(35)
    size = torch.exp2(low * torch.rand((2, 16, 128), generator=g, device="cuda"))
    size[:, ::2, ::2] *= 2.0 ** -10
    size[:, 1::2, 1::2] *= 2.0 ** -10
    case.q.copy_((torch.randn((2, 16, 128), generator=g, device="cuda") * size).to(case.q.dtype).view(2, -1))
    ws = case.workspace()
    case.run(ws)
    check(case)


@pytest.mark.parametrize("dim,group_size", [(128, -1), (128, 64), (64, -1), (256, 128)])
def test_long_sums_lean_to_neither_side(w4, dim, group_size):  # noqa: F811
    """The mean error of the outputs over a long sequence, at even and at odd places (whose codes go in at other sizes).

    Weights within 2^5 of one another in any 32 positions: products of codes (4 bits from 2^-22) and first parts of p s (11 bits) are multiples of
    2^-32 2^-5 = 2^-37 of the largest, which 24 bits from 2^-14 of it hold, so their sums are exact, and the remainders' are cut
    2^-11 below.  What is left are roundings to nearest, of fp32 and of the outputs: the latter, spread evenly over half a
    unit each, have a mean square of (2^-11 out)^2 / 3 at most, and their mean over N outputs a standard deviation of
    2^-11 rms(out) / sqrt(3 N).  Five of these are allowed.
    """
    import torch
    case = Case(w4, 36, "fp16", [131071], 32, 8, dim, 64, group_size, q_sigma=0.3)
    ws = case.workspace()
    case.run(ws)
    torch.cuda.synchronize()
    codes, params = (x.flatten(1, 2) for x in kv4.read(case.cache, 64, 8, dim, group_size, "fp16"))
    at, off, ref = case.slots[0], [], []
    for c in range(8):
        k, v = (kv4.values(codes[s][at, c], params[s][at, c]) for s in range(2))
        q = case.q[0].view(8, 4, dim)[c].double()
        p = torch.softmax(q @ k.t() * case.scale, -1)
        ref.append(p @ v)
        off.append(case.out[0].view(8, 4, dim)[c].double() - ref[-1])
        near = p[:, :131040].unflatten(-1, (-1, 32))
        assert float((near.amax(-1) / near.amin(-1)).max()) < 2.0 ** 5
    off, ref = torch.cat(off), torch.cat(ref)
    for place in range(2):
        x = off[:, place::2]
        limit = 5 * 2.0 ** -11 * float(ref.pow(2).mean().sqrt()) / (3 * x.numel()) ** 0.5
        assert abs(float(x.mean())) <= limit, (place, float(x.mean()) / limit)
