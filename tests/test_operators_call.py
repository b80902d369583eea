"""How the decode-step operators take their arguments from Python: the extension module and ctypes give
the same statuses for the same calls.  The pointers are fake, so every call here must be one that the
argument checks refuse, wherever the test runs: the statuses are written out, none is an error of a
missing GPU."""
import os

import numpy as np
import pytest

NAMES = ("w4a16_rope_append", "w4a16_paged_attention", "w4a16_moe_layer")
P = 0x10000
GOOD = {  # complete calls of each entry, of which a test spoils one argument
    "w4a16_rope_append": [P, 1024, P, 1024, P, 1024, P, 512, P, P, 4096, 256, 128, P, 100, P, 4, P, None, 4, 4, 2, 128,
                          128, None, 1, 16, 8, 0, 0],
    "w4a16_paged_attention": [P, 512, P, P, 4096, 256, 128, P, 512, None, P, 8, P, P, 1 << 30, 4, 4, 2, 128, 16, 8, 8,
                              0, 0.1, 0, 0],
    "w4a16_moe_layer": [P, 256, P, P, P, None, P, P, None, None, 256, P, 256, None, None, P, 1 << 30, 1, 256, 128, 8,
                        2, 64, 5, (1 << 14), 0],
}


@pytest.fixture(scope="module")
def w4():
    import weight_only_int4_03_gb300 as w4
    return w4


@pytest.fixture(scope="module")
def calls(w4):
    if not os.path.exists(w4.CALL_PATH):
        pytest.skip("built without Python's headers")
    return dict(zip(NAMES, (w4._rope_append, w4._paged_attention, w4._moe_layer)))


def args_of(name, **at):
    a = list(GOOD[name])
    sec = np.array([64], np.int32)
    if name == "w4a16_rope_append":
        a[24] = sec.ctypes.data
    for i, v in at.items():
        a[int(i[1:])] = v
    return a, sec


NULL, ALIGN, SHAPE, FLAGS, WORKSPACE, GROUP, TYPE = ((1 << 16) | d for d in (1, 2, 3, 4, 6, 7, 8))
UNSUPPORTED_SHAPE = (2 << 16) | 3
SPOILED = [
    ("w4a16_rope_append", dict(a28=8), FLAGS), ("w4a16_rope_append", dict(a19=-1), SHAPE),
    ("w4a16_rope_append", dict(a0=None), NULL), ("w4a16_rope_append", dict(a13=P + 2), ALIGN),
    ("w4a16_rope_append", dict(a11=-1), SHAPE),
    ("w4a16_paged_attention", dict(a24=8), FLAGS), ("w4a16_paged_attention", dict(a7=None), NULL),
    ("w4a16_paged_attention", dict(a18=127), UNSUPPORTED_SHAPE), ("w4a16_paged_attention", dict(a19=0), SHAPE),
    ("w4a16_moe_layer", dict(a23=4), FLAGS), ("w4a16_moe_layer", dict(a0=P + 2), ALIGN),
    ("w4a16_moe_layer", dict(a16=0), WORKSPACE), ("w4a16_moe_layer", dict(a17=65), UNSUPPORTED_SHAPE),
    ("w4a16_moe_layer", dict(a22=48), GROUP),
]


@pytest.mark.parametrize("name,spoil,want", SPOILED, ids=lambda v: str(v))
def test_both_ways_give_the_same_status(w4, calls, name, spoil, want):
    a, _keep = args_of(name, **spoil)
    assert getattr(w4._lib, name)(*a) == want
    assert calls[name](*a) == want
    assert w4._through_ctypes(name)(*a) == want


class FakeTensor:
    def __init__(self, address):
        self.address = address

    def data_ptr(self):
        return self.address


def test_pointers_from_tensors_and_arrays(w4, calls):
    table = np.zeros(64, np.float32)
    for call in (calls["w4a16_rope_append"], w4._through_ctypes("w4a16_rope_append")):
        a, _keep = args_of("w4a16_rope_append", a0=FakeTensor(P + 1))
        assert call(*a) == ALIGN
        a, _keep = args_of("w4a16_rope_append", a0=FakeTensor(0))
        assert call(*a) == NULL
        a, _keep = args_of("w4a16_rope_append", a13=table.view(np.uint8)[2:])  # two bytes past an aligned start
        assert call(*a) == ALIGN


def test_arguments_that_do_not_convert(calls):
    call = calls["w4a16_rope_append"]
    a, _keep = args_of("w4a16_rope_append")
    with pytest.raises(TypeError):
        call(*a[:-1])
    with pytest.raises(OverflowError):
        call(*args_of("w4a16_rope_append", a19=1 << 31)[0])
    with pytest.raises(OverflowError):
        call(*args_of("w4a16_rope_append", a28=-1)[0])
    with pytest.raises(TypeError):
        call(*args_of("w4a16_rope_append", a19=4.0)[0])
    with pytest.raises(AttributeError):
        call(*args_of("w4a16_rope_append", a0="q")[0])
    with pytest.raises(OverflowError):
        calls["w4a16_paged_attention"](*args_of("w4a16_paged_attention", a14=-1)[0])


def test_wrapper_raises_the_library_error(w4):
    with pytest.raises(w4.W4A16Error) as e:
        w4.w4a16_rope_append(P, P, P, P, P, P, P, P, P, None, 4, 4, 2, 128, 128, [60], 100, 16, 8, stream=0)
    assert e.value.status == (1 << 16) | 3


def outcome(call, args):
    try:
        return call(*args)
    except Exception as e:
        return type(e)


class Whole:
    def __index__(self):
        return 63


@pytest.mark.parametrize("name,spoil,want", [
    # numpy's scalars and whatever counts as an integer or a number
    ("w4a16_rope_append", dict(a23=np.int64(63)), SHAPE), ("w4a16_rope_append", dict(a23=np.uint8(63)), SHAPE),
    ("w4a16_rope_append", dict(a23=Whole()), SHAPE), ("w4a16_rope_append", dict(a28=True, a23=63), FLAGS),
    ("w4a16_paged_attention", dict(a23=np.float32(0.5), a24=8), FLAGS),
    ("w4a16_paged_attention", dict(a23=np.int32(1), a24=8), FLAGS),
    ("w4a16_paged_attention", dict(a23=1, a14=np.int64(0), a24=8), FLAGS),
    # what a parameter does not hold (in calls that are refused for another reason, were it taken)
    ("w4a16_rope_append", dict(a23=63, a19=(1 << 32) - 1), OverflowError),
    ("w4a16_rope_append", dict(a23=63, a28=1 << 32), OverflowError),
    ("w4a16_rope_append", dict(a23=63, a28=np.int64(-1)), OverflowError),
    ("w4a16_rope_append", dict(a23=63, a10=1 << 63), OverflowError),
    ("w4a16_rope_append", dict(a23=63, a0=1 << 64), OverflowError),
    ("w4a16_rope_append", dict(a23=63, a0=-(1 << 63) - 1), OverflowError),
    ("w4a16_paged_attention", dict(a14=1 << 64, a24=8), OverflowError),
    ("w4a16_paged_attention", dict(a14=-1, a24=8), OverflowError),
    # what is no number, or no buffer
    ("w4a16_rope_append", dict(a23=63, a19=4.0), TypeError),
    ("w4a16_rope_append", dict(a23=63, a19=None), TypeError),
    ("w4a16_rope_append", dict(a23=63, a19="4"), TypeError),
    ("w4a16_paged_attention", dict(a23="0.1", a24=8), TypeError),
    ("w4a16_paged_attention", dict(a23=None, a24=8), TypeError),
    ("w4a16_rope_append", dict(a23=63, a0="q"), AttributeError),
    ("w4a16_rope_append", dict(a23=63, a0=0.5), AttributeError),
    ("w4a16_rope_append", dict(a23=63, a0=np.int64(P)), AttributeError),
    ("w4a16_moe_layer", dict(a0=np.float32(1), a22=48), AttributeError),
], ids=lambda v: str(v))
def test_both_ways_take_and_refuse_the_same(w4, calls, name, spoil, want):
    a, _keep = args_of(name, **spoil)
    assert outcome(calls[name], a) == want
    assert outcome(w4._through_ctypes(name), a) == want


@pytest.mark.parametrize("name", NAMES)
def test_both_ways_count_their_arguments(w4, calls, name):
    a, _keep = args_of(name)
    a[-2] = 1 << 30  # a flag that no entry has, whatever the count
    for args in (a[:-1], a + [0]):
        assert outcome(calls[name], args) is TypeError
        assert outcome(w4._through_ctypes(name), args) is TypeError


@pytest.mark.parametrize("sections,error", [([30.5, 33.5], TypeError), ([1 << 32, 64], OverflowError), (["64"], TypeError)])
def test_sections_are_32_bit_integers(w4, sections, error):
    """Not cut to them: 30 and 33 of 30.5 and 33.5, or 0 of 2^32, would be other axes."""
    with pytest.raises(error):  # the flag is one that no entry has
        w4.w4a16_rope_append(P, P, P, P, P, P, P, P, P, None, 4, 4, 2, 128, 128, sections, 100, 16, 8, flags=1 << 30, stream=0)
