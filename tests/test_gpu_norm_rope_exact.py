"""The normed appends bit for bit against w4a16_rope_append, and what they report."""
import pytest

from test_gpu_norm_rope import Case, w4  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


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
