"""The normed appends bit for bit against w4a16_rope_append, and what they report."""
import pytest

from test_gpu_norm_rope import Case, w4  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


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
