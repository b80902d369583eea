"""w4a16_sample: the exactness of a token's share, temperatures down to the smallest, masked rows that end anywhere."""
import pytest

from test_gpu_sample import ALL, Case, w4  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu


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
