"""w4a16_norm_rope_append and w4a16_kv4_append against their formulas in 64 bits.

Tolerance.  With a and b a pair after the norm: the sum of squares of up to 512 values carries at most 16 + 5 + 2
roundings, half of which reaches its root; rsqrt is good to 2 units, and two products follow: below
(12 + 4 + 2) 2^-24 < 2^-19.8 of a and b.  The rotation adds 2^-24 for each of two products and their sum.  So before
its rounding to 16 bits a result is off by at most E = 2^-19 (|a| + |b|); rounded, by u |result| + E more, u half
a step of the type (and fp16 2^-25 where its numbers are subnormal).  A code is then off the rounded quotient by
1/2 + E / s, with s and b as stored.  Values are coded from what is given, in steps that are exact or single IEEE
operations: bit for bit.
"""
import pytest

import kv4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import weight_only_int4_03_gb300 as w4
    return w4


class Case:
    def __init__(self, seed, dtype, tokens, heads, kv, dim, rot, sections, page, adjacent=False, q_norm=True,
                 k_norm=True, group_size=None, pad=0, sigma=1.0, skip=(), page_pad=0, shift=0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = kv4.TYPES[dtype]
        self.__dict__.update(dtype=dtype, tokens=tokens, heads=heads, kv=kv, dim=dim, rot=rot, page=page,
                             sections=tuple(sections), adjacent=adjacent, group_size=group_size, eps=1e-6)
        width = (heads + 2 * kv) * dim + pad
        base = torch.randn(tokens * width + shift, generator=g, device="cuda") * sigma
        self.qkv = base.to(dt)[shift:].view(tokens, width)
        weight = lambda: (1 + 0.3 * torch.randn(dim + shift, generator=g, device="cuda")).to(dt)[shift:]
        self.q_norm = weight() if q_norm else None
        self.k_norm = weight() if k_norm else None
        self.max_pos = 4096
        self.table = torch.randn((self.max_pos, max(rot, 1)), generator=g, device="cuda")
        self.positions = torch.randint(0, self.max_pos, (max(len(sections), 1), tokens), generator=g, device="cuda",
                                       dtype=torch.int32)
        self.n_pages = (tokens + page - 1) // page + 2
        self.slots = torch.randperm(self.n_pages * page, generator=g, device="cuda")[:tokens].contiguous()
        for t in skip:
            self.slots[t] = -1
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.q_out = torch.full((tokens, heads * dim + pad), 7.0, dtype=dt, device="cuda")
        if group_size is None:
            self.k_cache, self.v_cache = (torch.full((self.n_pages, page, kv, dim), 5.0, dtype=dt, device="cuda")
                                          for _ in range(2))
        else:
            self.k_out, self.v_out = (torch.full((tokens, kv * dim + pad), 9.0, dtype=dt, device="cuda")
                                      for _ in range(2))
            self.page_pad = page_pad

    def flags(self, w4):
        return (w4.W4A16_FLAG_BF16 if self.dtype == "bf16" else 0) | (w4.W4A16_FLAG_ROPE_ADJACENT if self.adjacent else 0)

    def run(self, w4, **kw):
        import torch
        qkv, ld = self.qkv, self.qkv.shape[1]
        h, d = self.heads, self.dim
        parts = [qkv, qkv[:, h * d:], qkv[:, (h + self.kv) * d:]]
        common = dict(ldq=ld, ldk=ld, ldv=ld, ldqo=self.q_out.shape[1], **kw)
        sizes = [self.tokens, h, self.kv, d, self.rot, self.sections, self.max_pos, self.page, self.n_pages]
        if self.group_size is None:
            w4.w4a16_norm_rope_append(*parts, self.q_norm, self.k_norm, self.eps, self.q_out, self.k_cache, self.v_cache,
                                      self.table, self.positions, self.slots, self.status, *sizes, self.flags(w4), **common)
            return
        if not hasattr(self, "cache"):
            record = w4.w4a16_kv4_record_bytes(self.page, d, self.group_size)
            self.cache = torch.full((self.n_pages, self.kv * record + self.page_pad), 0x5A, dtype=torch.uint8, device="cuda")
        w4.w4a16_kv4_append(*parts, self.q_norm, self.k_norm, self.eps, self.q_out, self.cache, self.table, self.positions,
                            self.slots, self.status, *sizes, self.group_size, self.flags(w4), k_out=self.k_out,
                            v_out=self.v_out, ldko=self.k_out.shape[1], ldvo=self.v_out.shape[1],
                            page_stride=self.cache.shape[1], **common)

    def turned(self, x, weight):
        """(result, |a| + |b| of each value's pair) in 64 bits."""
        import torch
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + self.eps) * weight.double()
        y, size, half = x.clone(), x.abs(), self.rot // 2
        i = 0
        for axis, count in enumerate(self.sections):
            rows = self.table[self.positions[axis].long()].double()
            for _ in range(count):
                c, s = rows[:, i, None], rows[:, half + i, None]
                p, r = (2 * i, 2 * i + 1) if self.adjacent else (i, half + i)
                y[..., p] = x[..., p] * c - x[..., r] * s
                y[..., r] = x[..., r] * c + x[..., p] * s
                both = (x[..., p].abs() + x[..., r].abs()) * torch.maximum(c.abs(), s.abs()).clamp(min=1)
                size[..., p] = both
                size[..., r] = both
                i += 1
        return y, size

    def close(self, got, ref, size):
        import torch
        tol = kv4.UNIT[self.dtype] * ref.abs() + 2.0 ** -18.9 * size + 2.0 ** -25
        err = (got.double() - ref).abs()
        assert bool((err <= tol).all()), f"{float((err - tol).max())} over, {int((err > tol).sum())} values"

    def check(self):
        import torch
        torch.cuda.synchronize()
        t, h, kv, d = self.tokens, self.heads, self.kv, self.dim
        x = self.qkv[:, :(h + 2 * kv) * d].reshape(t, h + 2 * kv, d)
        if h:
            self.close(self.q_out[:, :h * d].reshape(t, h, d), *self.turned(x[:, :h], self.q_norm))
            assert bool((self.q_out[:, h * d:] == 7).all())
        k, size = self.turned(x[:, h:h + kv], self.k_norm)
        v = x[:, h + kv:]
        live = self.slots >= 0
        at = self.slots[live]
        untouched = torch.ones(self.n_pages * self.page, dtype=torch.bool, device="cuda")
        untouched[at] = False
        if self.group_size is None:
            kc, vc = (c.view(-1, kv, d) for c in (self.k_cache, self.v_cache))
            self.close(kc[at], k[live], size[live])
            assert torch.equal(vc[at], v[live])
            assert bool((kc[untouched] == 5).all()) and bool((vc[untouched] == 5).all())
            return
        codes, params = kv4.read(self.cache, self.page, kv, d, self.group_size, self.dtype)
        stands = kv4.values(codes, params)
        assert bool((self.k_out[:, kv * d:] == 9).all()) and bool((self.v_out[:, kv * d:] == 9).all())
        outs = [o[:, :kv * d].reshape(t, kv, d) for o in (self.k_out, self.v_out)]
        codes, params, stands = (z.flatten(1, 2) for z in (codes, params, stands))
        for side in range(2):  # what the cache stands for, rounded once (after an fma in fp32)
            ref = stands[side][at]
            tol = kv4.UNIT[self.dtype] * ref.abs() * (1 + 2.0 ** -12) + 2.0 ** -25
            assert bool(((outs[side][live].double() - ref).abs() <= tol).all())
        want, want_params = kv4.coded(v, self.group_size, self.dtype)
        assert torch.equal(codes[1][at], want[live])
        assert torch.equal(params[1][at], want_params[live])
        groups = kv4.groups_of(d, self.group_size)
        xk, e = (z[live].unflatten(-1, (groups, -1)) for z in (k, 2.0 ** -18.9 * size))
        s, b = (params[0][at][..., i].double() for i in range(2))
        u, off = kv4.UNIT[self.dtype], e.amax(-1)
        lo, hi = xk.amin(-1), xk.amax(-1)
        tiny = 2.0 ** -25 if self.dtype == "fp16" else 2.0 ** -126
        assert bool(((b - lo).abs() <= u * lo.abs() + 1.01 * off + tiny).all())
        assert bool(((s - (hi - lo) / 15).abs() <= u * (hi - lo) / 15 + 0.14 * off + tiny).all())
        quotient = ((xk - b.unsqueeze(-1)) / s.unsqueeze(-1)).clamp(0, 15)
        code = codes[0][at].unflatten(-1, (groups, -1)).double()
        assert bool(((code - quotient).abs() <= 0.5 + 1.01 * e / s.unsqueeze(-1) + 2.0 ** -20).all())
        # Rows that no slot names hold what they held.
        assert bool((codes[0][untouched] == torch.tensor([10, 5] * (d // 2), device="cuda", dtype=torch.int32)).all())


def name(c):
    return (f"{c['dtype']}t{c['tokens']}h{c['heads']}kv{c['kv']}d{c['dim']}r{c['rot']}s{len(c['sections'])}"
            f"p{c['page']}{'a' if c.get('adjacent') else ''}g{c.get('group_size')}")


WIDE = [
    dict(dtype="fp16", tokens=1, heads=32, kv=8, dim=128, rot=128, sections=[64], page=16),
    dict(dtype="bf16", tokens=33, heads=5, kv=1, dim=64, rot=32, sections=[16], page=24, adjacent=True, pad=8, skip=(3, 32)),
    dict(dtype="fp16", tokens=70, heads=3, kv=3, dim=256, rot=256, sections=[16, 56, 56], page=8),
    dict(dtype="bf16", tokens=19, heads=7, kv=2, dim=128, rot=128, sections=[13, 51], page=16, k_norm=False),
    dict(dtype="fp16", tokens=257, heads=16, kv=4, dim=128, rot=64, sections=[5, 10, 10, 7], page=1, q_norm=False),
    dict(dtype="bf16", tokens=2, heads=0, kv=4, dim=128, rot=0, sections=[], page=16),
    dict(dtype="fp16", tokens=1200, heads=40, kv=8, dim=128, rot=128, sections=[64], page=64, sigma=30.0),
    dict(dtype="fp16", tokens=5, heads=300, kv=2, dim=64, rot=64, sections=[32], page=16),
]


@pytest.mark.parametrize("kw", WIDE + [
    dict(dtype="fp16", tokens=9, heads=4, kv=2, dim=96, rot=96, sections=[48], page=16),
    dict(dtype="bf16", tokens=9, heads=4, kv=2, dim=80, rot=32, sections=[16], page=16),
    dict(dtype="fp16", tokens=3, heads=2, kv=2, dim=512, rot=512, sections=[256], page=16),
    # sizes, strides or addresses without 16-byte copies
    dict(dtype="fp16", tokens=11, heads=3, kv=2, dim=100, rot=36, sections=[11, 7], page=5, adjacent=True),
    dict(dtype="bf16", tokens=21, heads=3, kv=2, dim=65, rot=64, sections=[32], page=16),
    dict(dtype="fp16", tokens=21, heads=3, kv=2, dim=128, rot=128, sections=[64], page=16, pad=1, skip=(0,)),
    dict(dtype="bf16", tokens=4, heads=3, kv=1, dim=128, rot=128, sections=[64], page=16, shift=1),
    dict(dtype="bf16", tokens=300, heads=2, kv=1, dim=7, rot=0, sections=[], page=16, q_norm=False),
], ids=name)
def test_norm_rope_matches_formula(w4, kw):
    case = Case(3, **kw)
    case.run(w4)
    case.check()
    assert int(case.status.item()) == 0


@pytest.mark.parametrize("group_size", [-1, 64, 128])
@pytest.mark.parametrize("kw", WIDE, ids=name)
def test_kv4_append_matches_formula(w4, kw, group_size):
    if group_size > kw["dim"]:
        pytest.skip("no such group")
    case = Case(4, **kw, group_size=group_size, page_pad=32 if kw["tokens"] == 70 else 0)
    case.run(w4)
    case.check()
    assert int(case.status.item()) == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_kv4_groups_of_no_range_and_without_finite_values(w4, dtype):
    """Constant groups, ranges that round to nothing, infinities and NaN, ranges beyond the type; ties of codes."""
    import torch
    case = Case(5, dtype, 12, 0, 2, 128, 0, [], 16, k_norm=False, group_size=64)
    x = case.qkv.view(12, 4, 128)
    x[0] = 0
    x[1] = 1.5
    x[2] = -3.0
    tiny = 2.0 ** -24 if dtype == "fp16" else 2.0 ** -133
    x[3, :, ::3] = tiny
    x[3, :, 1::3] = 0
    x[3, :, 2::3] = 3 * tiny
    big = torch.finfo(x.dtype).max
    x[4, 0, 5], x[4, 1, 70], x[4, 2, 3], x[4, 3, 127] = float("inf"), float("-inf"), float("nan"), float("nan")
    if dtype == "fp16":
        x[5, :, 0], x[5, :, 1] = big, -big
    # Multiples of half a step: every odd one lies on the middle between two codes.
    x[6] = (torch.arange(128, device="cuda") % 31).to(x.dtype) * 0.5
    x[7] = (torch.arange(128, device="cuda") % 31 - 15).to(x.dtype) * 0.25
    case.run(w4)
    torch.cuda.synchronize()
    codes, params = kv4.read(case.cache, 16, 2, 128, 64, dtype)
    codes, params = codes.flatten(1, 2)[:, case.slots], params.flatten(1, 2)[:, case.slots]
    bad = torch.zeros((2, 12, 2, 2), dtype=torch.bool, device="cuda")
    bad[0, 4, 0, 0] = bad[0, 4, 1, 1] = bad[1, 4, 0, 0] = bad[1, 4, 1, 1] = True
    assert torch.equal(torch.isnan(params.float()).all(-1), bad)
    assert torch.equal(torch.isnan(params.float()).any(-1), bad)
    for side in range(2):
        want, want_params = kv4.coded(x[:, 2 * side:2 * side + 2], 64, dtype)
        s = want_params[..., 0].float()
        if dtype == "bf16":
            want_params[..., 0][s < 2.0 ** -126] = 0
        fine = ~bad[side]
        assert torch.equal(params[side][fine], want_params[fine])
        keep = fine & (want_params[..., 0].float() > 0)
        assert torch.equal(codes[side].unflatten(-1, (2, 64))[keep], want.unflatten(-1, (2, 64))[keep])
        none = fine & ~keep
        assert bool((codes[side].unflatten(-1, (2, 64))[none] == 0).all())
    out = case.k_out.view(12, 2, 2, 64)
    assert torch.equal(torch.isnan(out).all(-1), bad[0]) and torch.equal(torch.isnan(out).any(-1), bad[0])


@pytest.mark.parametrize("group_size", [None, 64])
def test_bad_positions_and_slots_are_reported(w4, group_size):
    import torch
    case = Case(6, "fp16", 6, 4, 2, 128, 128, [32, 32], 16, group_size=group_size)
    case.positions[1, 2] = case.max_pos  # half of the pairs
    case.positions[0, 4] = -1
    case.slots[5] = case.n_pages * case.page
    good = Case(6, "fp16", 6, 4, 2, 128, 128, [32, 32], 16, group_size=group_size)
    case.run(w4)
    good.run(w4)
    torch.cuda.synchronize()
    assert int(case.status.item()) == w4.W4A16_DEV_POSITION | w4.W4A16_DEV_SLOT
    for t in (0, 1, 3, 5):
        assert torch.equal(case.q_out[t], good.q_out[t])
    q = case.q_out[2].view(4, 2, 64)  # axis 1 has pairs 32..63: values 32..63 and 96..127
    assert bool((q[:, :, 32:] == 7).all()) and torch.equal(q[:, :, :32], good.q_out[2].view(4, 2, 64)[:, :, :32])
    if group_size is None:
        rows, same = case.k_cache.view(-1, 2, 128), good.k_cache.view(-1, 2, 128)
        assert bool((rows[good.slots[2]].view(2, 2, 64)[:, :, 32:] == 5).all())
        assert torch.equal(case.v_cache.view(-1, 2, 128)[good.slots[:5]], good.v_cache.view(-1, 2, 128)[good.slots[:5]])
        assert torch.equal(rows[good.slots[[0, 1, 3]]], same[good.slots[[0, 1, 3]]])
        assert bool((rows[good.slots[5]] == 5).all())
    else:
        a, b = (kv4.read(c.cache, 16, 2, 128, 64, "fp16")[0].flatten(1, 2) for c in (case, good))
        old = torch.tensor([10, 5] * 64, device="cuda", dtype=torch.int32)
        for t in range(6):
            slot = good.slots[t]
            assert torch.equal(a[1][slot], b[1][slot]) if t < 5 else bool((a[1][slot] == old).all())
            assert torch.equal(a[0][slot], b[0][slot]) if t in (0, 1, 3) else bool((a[0][slot] == old).all())
        assert bool((case.k_out[[2, 4]] == 9).all()) and torch.equal(case.k_out[5], good.k_out[5])
        assert torch.equal(case.v_out, good.v_out)


@pytest.mark.parametrize("group_size", [None, -1])
def test_in_place_side_stream_graph_and_repeats(w4, group_size):
    """q_out is q (and k_out, v_out are k, v); a captured call replayed on other inputs."""
    import torch
    kw = dict(dtype="bf16", tokens=40, heads=8, kv=2, dim=128, rot=128, sections=[64], page=16, group_size=group_size)
    want, case = Case(7, **kw), Case(7, **kw)
    want.run(w4)
    kept = case.qkv.clone()
    qkv, d = case.qkv, 128
    ld = qkv.shape[1]
    case.cache = torch.zeros_like(want.cache) if group_size else None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call():
        parts = [qkv, qkv[:, 8 * d:], qkv[:, 10 * d:]]
        sizes = [40, 8, 2, d, 128, (64,), case.max_pos, 16, case.n_pages]
        if group_size is None:
            w4.w4a16_norm_rope_append(*parts, case.q_norm, case.k_norm, case.eps, qkv, case.k_cache, case.v_cache, case.table,
                                      case.positions, case.slots, None, *sizes, case.flags(w4), ldq=ld, ldk=ld, ldv=ld,
                                      ldqo=ld, stream=side)
        else:
            w4.w4a16_kv4_append(*parts, case.q_norm, case.k_norm, case.eps, qkv, case.cache, case.table, case.positions,
                                case.slots, None, *sizes, group_size, case.flags(w4), k_out=parts[1], v_out=parts[2],
                                ldq=ld, ldk=ld, ldv=ld, ldqo=ld, ldko=ld, ldvo=ld, stream=side)

    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
        qkv.zero_()
        graph.replay()
        for _ in range(2):
            qkv.copy_(kept)
            graph.replay()
    side.synchronize()
    assert torch.equal(qkv[:, :8 * d], want.q_out)
    if group_size is None:
        assert torch.equal(case.k_cache, want.k_cache) and torch.equal(case.v_cache, want.v_cache)
    else:
        assert torch.equal(qkv[:, 8 * d:10 * d], want.k_out) and torch.equal(qkv[:, 10 * d:], want.v_out)
        a, b = (kv4.read(c, 16, 2, d, -1, "bf16") for c in (case.cache, want.cache))
        for x, y in zip(a, b):
            assert torch.equal(x.flatten(1, 2)[:, case.slots], y.flatten(1, 2)[:, case.slots])


def test_norm_of_one_is_the_rotary_append(w4):
    """Without weights the 16-bit entry gives the bits of w4a16_rope_append."""
    import torch
    case = Case(8, "fp16", 50, 8, 2, 128, 128, [64], 16, q_norm=False, k_norm=False)
    case.run(w4)
    q, k, v = torch.zeros_like(case.q_out), torch.full_like(case.k_cache, 5.0), torch.full_like(case.v_cache, 5.0)
    ld = case.qkv.shape[1]
    w4.w4a16_rope_append(case.qkv, case.qkv[:, 1024:], case.qkv[:, 1280:], q, k, v, case.table, case.positions, case.slots,
                         None, 50, 8, 2, 128, 128, [64], case.max_pos, 16, case.n_pages, ldq=ld, ldk=ld, ldv=ld)
    torch.cuda.synchronize()
    assert torch.equal(q, case.q_out) and torch.equal(k, case.k_cache) and torch.equal(v, case.v_cache)


def test_largest_prompt_side_by_side_tokens(w4):
    """More tokens than threads walk at once, and an offset into the cache that passes 32 bits."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(9)
    tokens, page, n_pages, kv, dim = 3000, 64, 1000, 2, 128
    record = w4.w4a16_kv4_record_bytes(page, dim, -1)
    stride = 5 * 2 ** 20  # pages of many layers: the last begins past 2^32
    cache = torch.zeros(n_pages * stride, dtype=torch.uint8, device="cuda").view(n_pages, stride)
    k, v = (torch.randn((tokens, kv, dim), generator=g, device="cuda").half() for _ in range(2))
    slots = torch.arange(n_pages * page - tokens, n_pages * page, device="cuda")
    w4.w4a16_kv4_append(None, k, v, None, None, 0.0, None, cache, None, None, slots, None, tokens, 0, kv, dim, 0, (), 0,
                        page, n_pages, -1, page_stride=stride)
    torch.cuda.synchronize()
    first = (n_pages * page - tokens) // page
    codes, params = kv4.read(cache[first:, :kv * record].contiguous(), page, kv, dim, -1, "fp16")
    at = slots - first * page
    want, want_params = kv4.coded(v, -1, "fp16")
    assert torch.equal(codes.flatten(1, 2)[1][at], want) and torch.equal(params.flatten(1, 2)[1][at], want_params)
    want, want_params = kv4.coded(k, -1, "fp16")
    assert torch.equal(codes.flatten(1, 2)[0][at], want) and torch.equal(params.flatten(1, 2)[0][at], want_params)
