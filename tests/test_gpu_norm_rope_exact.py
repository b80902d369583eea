"""The normed appends bit for bit: key codes against 64 bits, the 16-bit entry against w4a16_rope_append; reports.

Keys are coded from two-part results.  Base and step are those of exact arithmetic rounded to fp32 and then to 16 bits: a
part of 2^-46 is what they could be off by, which no group of a test meets.  A code comes from the remainder r z - (b + q s),
in three fma's of numbers below s / 2 (each off by at most half a unit of these, 2^-25 s), and a quotient off by as much.  A
key falls on the other side of a border where its error reaches it: the chance of that is the mean size of the error in
steps, which for four errors spread evenly over their ranges is at most sqrt(4 / 3) 2^-25.  With N keys n = N sqrt(4 / 3) 2^-25
of them are expected, and n + 5 sqrt(n) allowed (5 standard deviations of a count).  In fp32 alone more are wrong, and bases and
steps too: the test counts these in the reference, to show that it would see them.
"""
import pytest

import kv4
from test_gpu_norm_rope import Case, w4  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


def near_a_border(x, dtype):
    """Numbers that fp32's errors could take to another 16-bit number: within 2^-22 of the middle between two."""
    import torch
    bits = {"fp16": 10, "bf16": 7}[dtype]
    scaled = x.abs() / torch.exp2(torch.floor(torch.log2(x.abs()))) * 2 ** bits
    return ((scaled - scaled.floor() - 0.5).abs() < 2.0 ** (bits - 22)) & (x != 0)


def turned_in_fp32(case, x):
    import torch
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + case.eps) * case.k_norm.float()
    half = case.rot // 2
    axis = torch.repeat_interleave(torch.arange(len(case.sections)), torch.tensor(case.sections)).cuda()
    at, pair = case.positions.long()[axis].t(), torch.arange(half, device="cuda")
    c, s = case.table[at, pair][:, None], case.table[at, half + pair][:, None]
    first, second = ((slice(0, case.rot, 2), slice(1, case.rot, 2)) if case.adjacent else
                     (slice(0, half), slice(half, case.rot)))
    y = x.clone()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


@pytest.mark.parametrize("dtype,dim,group_size,rot,sections,adjacent", [
    ("bf16", 64, -1, 64, [32], False), ("fp16", 128, 64, 128, [16, 24, 24], False), ("bf16", 128, 64, 128, [16, 24, 24], True),
    ("fp16", 128, -1, 64, [32], True), ("bf16", 256, 64, 256, [128], False), ("fp16", 256, 128, 128, [64], False),
    ("bf16", 128, 64, 0, [], False),
])
def test_key_codes_are_those_of_64_bits(w4, dtype, dim, group_size, rot, sections, adjacent):  # noqa: F811
    import torch
    keys = wrong = doubtful = in_fp32 = params_in_fp32 = 0
    for seed in range(12):
        case = Case(100 + seed, dtype, 2 ** 23 // (4 * dim), 1, 4, dim, rot, sections, 32, adjacent=adjacent,
                    group_size=group_size)
        if rot:  # angles, not any numbers
            angle = torch.rand((case.max_pos, rot // 2), device="cuda", dtype=torch.float64,
                               generator=torch.Generator(device="cuda").manual_seed(seed)) * 6.3
            case.table = torch.cat((angle.cos(), angle.sin()), 1).float().contiguous()
        case.run(w4)
        torch.cuda.synchronize()
        codes, params = (x.flatten(1, 2)[0][case.slots] for x in kv4.read(case.cache, 32, 4, dim, group_size, dtype))
        x = case.qkv.view(case.tokens, 9, dim)[:, 1:5]
        k, _ = case.turned(x, case.k_norm)
        k = k.unflatten(-1, (kv4.groups_of(dim, group_size), -1))
        lo, hi = k.amin(-1), k.amax(-1)
        step = (hi - lo) / 15
        b, s = (y.float().to(kv4.TYPES[dtype]) for y in (lo, step))
        assert torch.equal(params[..., 0], s) and torch.equal(params[..., 1], b)
        if rot:
            plain = turned_in_fp32(case, x).unflatten(-1, k.shape[-2:])
        want = ((k - b.double().unsqueeze(-1)) / s.double().unsqueeze(-1)).round().clamp(0, 15).int()
        wrong += int((codes.unflatten(-1, want.shape[-2:]) != want).sum())
        if rot:
            low, high = plain.amin(-1), plain.amax(-1)
            params_in_fp32 += sum(int((y.to(z.dtype) != z).sum()) for y, z in ((low, b), ((high - low) / 15, s)))
            in_fp32 += int((((plain - b.float().unsqueeze(-1)) / s.float().unsqueeze(-1)).round().clamp(0, 15) != want).sum())
        doubtful += int(near_a_border(lo, dtype).sum()) + int(near_a_border(step, dtype).sum())
        keys += want.numel()
    expected = keys * (4 / 3) ** 0.5 * 2.0 ** -25
    most = expected + 5 * expected ** 0.5
    print(f"{wrong} of {keys} codes ({in_fp32} in fp32, {most:.0f} at most), {doubtful} bases and steps near a border "
          f"({params_in_fp32} wrong in fp32)")
    assert wrong <= most
    assert doubtful >= 10 and (not rot or (in_fp32 > most and params_in_fp32 > 0))


FORMS = [
    dict(tokens=50, heads=8, kv=2, dim=128, rot=128, sections=[64]),
    dict(tokens=1500, heads=8, kv=2, dim=128, rot=128, sections=[64]),                    # a prompt
    dict(tokens=1500, heads=8, kv=2, dim=128, rot=128, sections=[64], adjacent=True),
    dict(tokens=40, heads=4, kv=1, dim=64, rot=32, sections=[16], adjacent=True),
    dict(tokens=1100, heads=4, kv=2, dim=256, rot=128, sections=[13, 30, 21]),             # cuts inside eight pairs
    dict(tokens=1100, heads=4, kv=2, dim=128, rot=128, sections=[13, 30, 21], adjacent=True),
    dict(tokens=60, heads=3, kv=2, dim=100, rot=36, sections=[11, 7]),                     # without 16-byte copies
    dict(tokens=60, heads=3, kv=2, dim=100, rot=36, sections=[11, 7], adjacent=True),
    dict(tokens=900, heads=5, kv=3, dim=128, rot=128, sections=[64], pad=1),
    dict(tokens=30, heads=5, kv=3, dim=128, rot=64, sections=[32], shift=1, skip=(4,)),
    dict(tokens=300, heads=3, kv=1, dim=576, rot=576, sections=[288]),                     # heads wider than 512
    dict(tokens=300, heads=3, kv=1, dim=1024, rot=64, sections=[5, 27], adjacent=True),
    dict(tokens=300, heads=3, kv=1, dim=576, rot=64, sections=[32], pad=1),
]


@pytest.mark.parametrize("kw", FORMS, ids=lambda c: f"t{c['tokens']}d{c['dim']}r{c['rot']}s{len(c['sections'])}"
                         f"{'a' if c.get('adjacent') else ''}{'u' if c.get('pad') or c.get('shift') else ''}")
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_without_weights_the_bits_of_the_rotary_append(w4, dtype, kw):  # noqa: F811
    import torch
    case = Case(8, dtype, page=16, q_norm=False, k_norm=False, **kw)
    case.run(w4)
    q, k, v = torch.full_like(case.q_out, 7.0), torch.full_like(case.k_cache, 5.0), torch.full_like(case.v_cache, 5.0)
    ld, h, kv, d = case.qkv.shape[1], case.heads, case.kv, case.dim
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w4.w4a16_rope_append(case.qkv, case.qkv[:, h * d:], case.qkv[:, (h + kv) * d:], q, k, v, case.table, case.positions,
                         case.slots, status, case.tokens, h, kv, d, case.rot, case.sections, case.max_pos, 16, case.n_pages,
                         case.flags(w4), ldq=ld, ldk=ld, ldv=ld, ldqo=q.shape[1])
    torch.cuda.synchronize()
    assert torch.equal(v, case.v_cache)
    assert torch.equal(q, case.q_out), int((q != case.q_out).sum())
    assert torch.equal(k, case.k_cache), int((k != case.k_cache).sum())
    assert int(case.status.item()) == 0 and int(status.item()) == 0


@pytest.mark.parametrize("pad", [0, 1], ids=["wide", "any"])
@pytest.mark.parametrize("heads", [0, 2])
@pytest.mark.parametrize("slot", [-1, "past"])
def test_positions_of_tokens_without_a_slot_are_reported(w4, slot, heads, pad):  # noqa: F811
    """As w4a16_rope_append does, whichever kernel a call takes."""
    import torch
    case = Case(9, "fp16", 5, heads, 2, 128, 128, [32, 32], 16, pad=pad)
    case.positions[1, 3] = case.max_pos + 7
    case.slots[3] = -1 if slot == -1 else case.n_pages * 16
    case.run(w4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ld, d = case.qkv.shape[1], 128
    w4.w4a16_rope_append(case.qkv, case.qkv[:, heads * d:], case.qkv[:, (heads + 2) * d:], case.q_out.clone(),
                         case.k_cache.clone(), case.v_cache.clone(), case.table, case.positions, case.slots, status, 5, heads,
                         2, d, d, [32, 32], case.max_pos, 16, case.n_pages, ldq=ld, ldk=ld, ldv=ld, ldqo=case.q_out.shape[1])
    torch.cuda.synchronize()
    want = w4.W4A16_DEV_POSITION | (0 if slot == -1 else w4.W4A16_DEV_SLOT)
    assert int(status.item()) == want and int(case.status.item()) == want
