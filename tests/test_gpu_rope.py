"""w4a16_rope_append against its formula in 64 bits.

Tolerance: two fp32 products and a sum (relative error 2^-22 of |x1 c| + |x2 s|), then one rounding
to the output type with unit roundoff u (2^-11 fp16, 2^-8 bf16): u |ref| + 2^-21 (|x1| + |x2|).  Copied values
and v are compared bit for bit.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

UNIT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def w4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import weight_only_int4_03_gb300 as w4
    return w4


def dtype_of(name):
    import torch
    return torch.float16 if name == "fp16" else torch.bfloat16


class Case:
    def __init__(self, seed, dtype, tokens, heads, kv, dim, rot, sections, page, adjacent=False, max_pos=500,
                 pad=0, order="token"):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = dtype_of(dtype)
        self.__dict__.update(dtype=dtype, tokens=tokens, heads=heads, kv=kv, dim=dim, rot=rot,
                             sections=sections, page=page, adjacent=adjacent, max_pos=max_pos)
        self.ld = (heads + 2 * kv) * dim + pad
        self.qkv = torch.randn((tokens, self.ld), generator=g, device="cuda", dtype=dt)
        self.table = torch.randn((max_pos, rot), generator=g, device="cuda")
        self.positions = torch.randint(0, max_pos, (len(sections), tokens), generator=g, device="cuda",
                                       dtype=torch.int32)
        self.n_pages = (tokens + page - 1) // page + 2
        self.slots = torch.randperm(self.n_pages * page, generator=g, device="cuda")[:tokens].contiguous()
        if order == "token":   # [page][token][head][dim]
            shape, self.strides = (self.n_pages, page, kv, dim), None
        else:                  # [page][head][token][dim]
            shape, self.strides = (self.n_pages, kv, page, dim), (kv * page * dim, dim, page * dim)
        self.order = order
        self.k_cache = torch.randn(shape, generator=g, device="cuda", dtype=dt)
        self.v_cache = torch.randn(shape, generator=g, device="cuda", dtype=dt)
        self.q_out = torch.full((tokens, heads, dim), float("nan"), device="cuda", dtype=dt)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def parts(self):
        h, k, d = self.heads, self.kv, self.dim
        return self.qkv, self.qkv[:, h * d:], self.qkv[:, (h + k) * d:]

    def run(self, w4, q_out=None, ldqo=None, **kw):
        flags = (w4.W4A16_FLAG_BF16 if self.dtype == "bf16" else 0) | (
            w4.W4A16_FLAG_ROPE_ADJACENT if self.adjacent else 0)
        q, k, v = self.parts()
        w4.w4a16_rope_append(q, k, v, self.q_out if q_out is None else q_out, self.k_cache, self.v_cache,
                             self.table, self.positions, self.slots, self.status, self.tokens, self.heads,
                             self.kv, self.dim, self.rot, self.sections, self.max_pos, self.page, self.n_pages,
                             flags, ldq=self.ld, ldk=self.ld, ldv=self.ld, ldqo=ldqo, kv_strides=self.strides, **kw)

    def rows(self, cache):
        """A cache as [slot][head][dim]."""
        if self.order != "token":
            cache = cache.transpose(1, 2)
        return cache.reshape(-1, self.kv, self.dim)

    def reference(self):
        """(q and k turned [t, heads + kv, dim] in fp64, tolerance, v's bits)."""
        import torch
        t, h, k, d, half = self.tokens, self.heads, self.kv, self.dim, self.rot // 2
        x = self.qkv[:, :(h + 2 * k) * d].reshape(t, h + 2 * k, d).double()
        y = x[:, :h + k].clone()
        tol = torch.zeros_like(y)
        i = 0
        for axis, count in enumerate(self.sections):
            row = self.table[self.positions[axis].long()].double()
            for _ in range(count):
                c, s = row[:, i, None], row[:, half + i, None]
                a, b = (2 * i, 2 * i + 1) if self.adjacent else (i, half + i)
                x1, x2 = x[:, :h + k, a], x[:, :h + k, b]
                y[:, :, a] = x1 * c - x2 * s
                y[:, :, b] = x2 * c + x1 * s
                mag = (x1.abs() + x2.abs()) * (c.abs() + s.abs())
                tol[:, :, a] = UNIT[self.dtype] * y[:, :, a].abs() + 2.0 ** -21 * mag
                tol[:, :, b] = UNIT[self.dtype] * y[:, :, b].abs() + 2.0 ** -21 * mag
                i += 1
        return y, tol + 1e-30, x[:, h + k:]


def check(case, q_out, before_k, before_v):
    import torch
    y, tol, v = case.reference()
    torch.cuda.synchronize()
    h = case.heads
    # fp16 subnormals have a fixed spacing: half of 2^-24.
    tol = tol + (2.0 ** -25 if case.dtype == "fp16" else 0.0)
    tol[..., case.rot:] = 0.0
    assert bool(((q_out.double() - y[:, :h]).abs() <= tol[:, :h]).all())
    live = case.slots >= 0
    kr, vr = case.rows(case.k_cache), case.rows(case.v_cache)
    assert bool(((kr[case.slots[live]].double() - y[live, h:]).abs() <= tol[live, h:]).all())
    assert bool((vr[case.slots[live]].double() == v[live]).all())
    other = torch.ones(kr.shape[0], dtype=torch.bool, device="cuda")
    other[case.slots[live]] = False
    assert torch.equal(kr[other], case.rows(before_k)[other])  # no other row is touched
    assert torch.equal(vr[other], case.rows(before_v)[other])
    assert int(case.status.item()) == 0


CASES = [
    dict(dtype="fp16", tokens=1, heads=32, kv=8, dim=128, rot=128, sections=[64], page=16),
    dict(dtype="bf16", tokens=7, heads=5, kv=1, dim=64, rot=32, sections=[16], page=24, adjacent=True),
    dict(dtype="bf16", tokens=130, heads=6, kv=2, dim=128, rot=128, sections=[16, 24, 24], page=16),
    dict(dtype="fp16", tokens=33, heads=3, kv=3, dim=96, rot=48, sections=[5, 12, 7], page=8),
    dict(dtype="fp16", tokens=33, heads=3, kv=3, dim=96, rot=48, sections=[5, 0, 12, 7], page=8, adjacent=True),
    dict(dtype="bf16", tokens=9, heads=4, kv=2, dim=256, rot=256, sections=[1, 127], page=1),
    dict(dtype="fp16", tokens=19, heads=2, kv=1, dim=80, rot=20, sections=[3, 7], page=5),     # any-size path
    dict(dtype="bf16", tokens=19, heads=2, kv=1, dim=33, rot=6, sections=[1, 1, 1], page=5, adjacent=True),
    dict(dtype="fp16", tokens=12, heads=2, kv=2, dim=64, rot=64, sections=[32], page=16, pad=3),  # odd stride
    dict(dtype="bf16", tokens=40, heads=4, kv=4, dim=64, rot=64, sections=[32], page=16, order="head"),
    dict(dtype="fp16", tokens=700, heads=40, kv=8, dim=128, rot=64, sections=[32], page=64),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda c: "-".join(str(v) for v in c.values()).replace(" ", ""))
def test_matches_formula(w4, kw):
    case = Case(1, **kw)
    before = case.k_cache.clone(), case.v_cache.clone()
    case.run(w4)
    check(case, case.q_out, *before)


def test_in_place_and_padding(w4):
    """q turned where it lies; negative slots leave the cache alone but their q is turned."""
    case = Case(2, "fp16", 21, 4, 2, 128, 128, [16, 24, 24], 16)
    case.slots[3] = -1
    case.slots[20] = -7
    before = case.k_cache.clone(), case.v_cache.clone()
    keep = case.qkv.clone()
    case.run(w4, q_out=case.qkv, ldqo=case.ld)
    got = case.qkv[:, :case.heads * case.dim].reshape(21, case.heads, case.dim).clone()
    assert (case.qkv[:, case.heads * case.dim:] == keep[:, case.heads * case.dim:]).all()
    case.qkv.copy_(keep)
    check(case, got, *before)


def test_only_q_and_only_kv(w4):
    import torch
    case = Case(3, "bf16", 10, 4, 2, 64, 64, [32], 16)
    before = case.k_cache.clone(), case.v_cache.clone()
    q, k, v = case.parts()
    args = (case.status, 10)
    w4.w4a16_rope_append(q, None, None, case.q_out, None, None, case.table, case.positions, None, *args, 4, 0, 64,
                         64, [32], case.max_pos, 1, 1, w4.W4A16_FLAG_BF16, ldq=case.ld)
    w4.w4a16_rope_append(None, k, v, None, case.k_cache, case.v_cache, case.table, case.positions, case.slots,
                         *args, 0, 2, 64, 64, [32], case.max_pos, 16, case.n_pages, w4.W4A16_FLAG_BF16,
                         ldk=case.ld, ldv=case.ld)
    torch.cuda.synchronize()
    check(case, case.q_out, *before)


@pytest.mark.parametrize("dim,rot", [(128, 128), (40, 12)])
def test_bad_positions_and_slots_are_reported(w4, dim, rot):
    """Out-of-range entries are skipped and reported; every other token is as ever."""
    import torch
    case = Case(4, "fp16", 12, 4, 2, dim, rot, [rot // 2], 8)
    good = Case(4, "fp16", 12, 4, 2, dim, rot, [rot // 2], 8)
    good.run(w4)
    case.positions[0, 2] = case.max_pos
    case.positions[0, 5] = -1
    case.slots[7] = case.n_pages * 8
    before = case.k_cache.clone()
    case.run(w4)
    torch.cuda.synchronize()
    assert int(case.status.item()) == w4.W4A16_DEV_POSITION | w4.W4A16_DEV_SLOT
    ok = [t for t in range(12) if t not in (2, 5)]
    assert torch.equal(case.q_out[ok], good.q_out[ok])
    assert bool(torch.isnan(case.q_out[[2, 5], :, :rot]).all())
    rows = [int(case.slots[t]) for t in ok if t != 7]
    assert torch.equal(case.rows(case.k_cache)[rows], good.rows(good.k_cache)[rows])
    bad = [int(good.slots[7])]
    assert torch.equal(case.rows(case.k_cache)[bad], case.rows(before)[bad])


def test_side_stream_and_graph(w4):
    import torch
    case = Case(5, "bf16", 64, 8, 2, 128, 128, [64], 16)
    before = case.k_cache.clone(), case.v_cache.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            case.run(w4, stream=side)
        graph.replay()
        graph.replay()
    side.synchronize()
    check(case, case.q_out, *before)


@pytest.mark.parametrize("heads", [1, 3, 5, 8])
@pytest.mark.parametrize("dim,rot", [(64, 64), (40, 12)])
def test_q_alone_looks_at_no_cache_argument(w4, heads, dim, rot):
    """Without KV heads the slots and the cache's sizes mean nothing, whatever the number of heads."""
    import torch
    case = Case(6, "fp16", 9, heads, 1, dim, rot, [rot // 2], 8)
    q = case.parts()[0]
    for slots in (None, torch.full((9,), 1 << 40, dtype=torch.int64, device="cuda")):
        case.q_out.fill_(float("nan"))
        w4.w4a16_rope_append(q, None, None, case.q_out, None, None, case.table, case.positions, slots, case.status, 9,
                             heads, 0, dim, rot, [rot // 2], case.max_pos, 1, 1, ldq=case.ld)
        torch.cuda.synchronize()
        y, tol, _ = case.reference()
        assert bool(((case.q_out.double() - y[:, :heads]).abs() <= tol[:, :heads] + 2.0 ** -25).all())
        assert int(case.status.item()) == 0


def test_as_many_tokens_as_an_int_counts(w4):
    """The walk over tokens ends at the last one, not past it: 2^31 - 1 rows of one narrow head, in place."""
    import torch
    torch.cuda.empty_cache()
    n, dim = (1 << 31) - 1, 16
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 80 GB")
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.zeros((n, dim), dtype=torch.float16, device="cuda")
    rows = torch.tensor([0, 1, 1 << 20, (1 << 31) - 250000, (1 << 31) - 120000, (1 << 31) - 116737, n - 116000, n - 2,
                         n - 1], device="cuda")
    x[rows] = torch.randn((rows.numel(), dim), generator=g, device="cuda", dtype=torch.float16)
    before = x[rows].double()
    table = torch.randn((2, dim), generator=g, device="cuda")
    positions = torch.ones(n, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w4.w4a16_rope_append(x, None, None, x, None, None, table, positions, None, status, n, 1, 0, dim, dim, [8], 2, 1, 1)
    torch.cuda.synchronize()
    c, s = table[1, :8].double(), table[1, 8:].double()
    a, b = before[:, :8], before[:, 8:]
    ref = torch.cat([a * c - b * s, b * c + a * s], 1)
    mag = (a.abs() + b.abs()) * (c.abs() + s.abs())
    tol = UNIT["fp16"] * ref.abs() + 2.0 ** -21 * torch.cat([mag, mag], 1) + 2.0 ** -25
    assert bool(((x[rows].double() - ref).abs() <= tol).all())
    assert int(status.item()) == 0
    del x, positions
    torch.cuda.empty_cache()
