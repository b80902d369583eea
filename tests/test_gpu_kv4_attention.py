"""w4a16_kv4_attention against its formula in 64 bits, over what the cache's codes, steps and bases stand for.

Tolerance.  A score is scale (s (q . c) + b sum q), its first part a chain of at most head_dim / 16 tensor-core sums,
each cut off at 2^-23, then four fp32 roundings: off by at most E = (D / 16 + 6) 2^-23 B with
B = scale max_i sum |q| (|s| c + |b|), taken from the data.  So p is off by a factor e^(2 E) at most (score and
maximum), and exp2 adds 2^-22.  p s goes on with 2^-22 of itself, in bf16 with 2^-11, times codes less 8, and a part's
sums (of codes less 8: at most 8 steps, and a + 8 s) are cut off at 2^-23 in six products of 32 positions and rounded at
2^-24 once for these; the joins add fewer.  With R the largest of |value| and 16 |s|, all of that is below
(4 E + 2^-17) R, and the rounding of bf16's p s below 2^-12 R (8 s is half of 16 s).  So
|out - ref| <= u |ref| + (4 E + 2^-17) R, plus 2^-12 R in bf16, with u half a step of the type, and
|lse - ref| <= E + 2^-20 + 2^-22 |ref|.
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
    """Sequences of the given lengths over shuffled pages; rows that no sequence owns hold steps and bases of NaN."""

    def __init__(self, w4, seed, dtype, lens, heads, kv, dim, page, group_size=-1, window=0, q_pad=0, o_pad=0,
                 table_pad=0, sigma=1.0, page_pad=0, offset=0.0, q_sigma=1.0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = kv4.TYPES[dtype]
        self.__dict__.update(w4=w4, dtype=dtype, lens_list=list(lens), heads=heads, kv=kv, dim=dim, page=page,
                             group_size=group_size, window=window, batch=len(lens), scale=dim ** -0.5)
        need = [(n + page - 1) // page for n in lens]
        self.n_pages = sum(need) + 2
        self.max_pages = max(max(need), 1)
        order = torch.randperm(self.n_pages, generator=g, device="cuda").to(torch.int32)
        # Unused table entries hold numbers that must not be looked up.
        self.table = torch.full((self.batch, self.max_pages + table_pad), -12345, dtype=torch.int32, device="cuda")
        record = w4.w4a16_kv4_record_bytes(page, dim, group_size)
        # 0x7F bytes everywhere: a step and base of 0x7F7F are NaN in both types.
        self.cache = torch.full((self.n_pages, kv * record + page_pad), 0x7F, dtype=torch.uint8, device="cuda")
        if dtype == "bf16":
            self.cache.fill_(0xFF)
        self.flags = w4.W4A16_FLAG_BF16 if dtype == "bf16" else 0
        at = 0
        slots = []
        for i, n in enumerate(lens):
            self.table[i, :need[i]] = order[at:at + need[i]]
            pos = torch.arange(n, device="cuda")
            slots.append(order[at:at + need[i]].long()[pos // page] * page + pos % page if n else pos)
            at += need[i]
        self.slots = slots
        every = torch.cat(slots)
        t = every.numel()
        size = torch.exp(0.3 * torch.randn((kv, dim), generator=g, device="cuda"))
        k = ((torch.randn((t, kv, dim), generator=g, device="cuda") * size + offset) * sigma).to(dt)
        v = (torch.randn((t, kv, dim), generator=g, device="cuda") * size + offset).to(dt)
        if t:
            w4.w4a16_kv4_append(None, k, v, None, None, 0.0, None, self.cache, None, None, every, None, t, 0, kv, dim, 0, (),
                                0, page, self.n_pages, group_size, self.flags, page_stride=self.cache.shape[1])
        self.q = (torch.randn((self.batch, heads * dim + q_pad), generator=g, device="cuda") * q_sigma).to(dt)
        self.out = torch.full((self.batch, heads * dim + o_pad), float("nan"), device="cuda", dtype=dt)
        self.lse = torch.full((self.batch, heads), float("nan"), device="cuda")
        self.lens = torch.tensor(self.lens_list, dtype=torch.int32, device="cuda")

    def workspace(self):
        import torch
        size = self.w4.w4a16_kv4_attention_workspace_size(self.batch, self.heads, self.kv, self.dim)
        assert size > 0
        return torch.zeros(size, dtype=torch.uint8, device="cuda")

    def run(self, ws, lse=True, **kw):
        self.w4.w4a16_kv4_attention(self.q, self.cache, self.out, self.table, self.lens, ws, self.batch, self.heads,
                                    self.kv, self.dim, self.page, self.n_pages, self.max_pages, self.group_size, self.scale,
                                    self.flags, window=self.window, lse=self.lse if lse else None, ldq=self.q.shape[1],
                                    ldo=self.out.shape[1], ld_table=self.table.shape[1], page_stride=self.cache.shape[1], **kw)

    def check(self, dead=()):
        """dead: (sequence, position) pairs that are masked."""
        import torch
        torch.cuda.synchronize()
        group = self.heads // self.kv
        codes, params = kv4.read(self.cache, self.page, self.kv, self.dim, self.group_size, self.dtype)
        codes, params = codes.flatten(1, 2), params.flatten(1, 2)
        for i, n in enumerate(self.lens_list):
            got = self.out[i, :self.heads * self.dim].view(self.heads, self.dim).double()
            first = max(0, n - self.window) if self.window else 0
            rows = [int(r) for r in range(first, n) if (i, r) not in dead] if dead else range(first, n)
            if not len(rows):
                assert bool((got == 0).all())
                assert bool((self.lse[i] == float("-inf")).all())
                continue
            at = self.slots[i][first:n] if not dead else self.slots[i][torch.tensor(rows, device="cuda")]
            sides = [kv4.values(codes[s][at], params[s][at]) for s in range(2)]
            q = self.q[i, :self.heads * self.dim].view(self.kv, group, self.dim).double()
            logits = torch.einsum("cgd,ncd->cgn", q, sides[0]) * self.scale
            ref = torch.einsum("cgn,ncd->cgd", torch.softmax(logits, -1), sides[1]).reshape(self.heads, self.dim)
            lse = torch.logsumexp(logits, -1).reshape(self.heads)
            s, b = (params[0][at][..., j].double() for j in range(2))
            weight = (codes[0][at].unflatten(-1, (s.shape[-1], -1)) * s.abs().unsqueeze(-1) + b.abs().unsqueeze(-1)).flatten(-2)
            bound = float((torch.einsum("cgd,ncd->cgn", q.abs(), weight) * self.scale).max())
            e = (self.dim / 16 + 6) * 2.0 ** -23 * bound
            r = max(float(sides[1].abs().max()), 16 * float(params[1][at][..., 0].double().abs().max()))
            part = 2.0 ** -17 + (2.0 ** -12 if self.dtype == "bf16" else 0.0)
            tol = kv4.UNIT[self.dtype] * ref.abs() + (4 * e + part) * r + 2.0 ** -25
            err = (got - ref).abs()
            assert bool((err <= tol).all()), f"sequence {i} (length {n}): {float((err / tol).max())} times the tolerance"
            off = (self.lse[i].double() - lse).abs()
            assert bool((off <= e + 2.0 ** -20 + 2.0 ** -22 * lse.abs()).all()), (i, float(off.max()), e)


CASES = [
    dict(dtype="fp16", lens=[1], heads=8, kv=2, dim=128, page=16),
    dict(dtype="bf16", lens=[37], heads=4, kv=4, dim=64, page=16),
    dict(dtype="fp16", lens=[0, 1, 15, 16, 17, 63, 64, 65, 0, 129], heads=16, kv=2, dim=128, page=16),
    dict(dtype="bf16", lens=[31, 32, 33, 127, 128, 129, 255, 257, 7, 8, 9], heads=8, kv=1, dim=128, page=8, group_size=64),
    dict(dtype="bf16", lens=[5, 300, 0, 2, 777], heads=12, kv=12, dim=64, page=24, table_pad=3),
    dict(dtype="fp16", lens=[4000], heads=5, kv=1, dim=128, page=64),
    dict(dtype="bf16", lens=[9001, 3], heads=40, kv=8, dim=128, page=32, group_size=64),
    dict(dtype="bf16", lens=[70, 1200], heads=9, kv=1, dim=128, page=8),          # nine heads: two tiles of columns
    dict(dtype="fp16", lens=[70, 1200], heads=32, kv=2, dim=64, page=8),          # sixteen
    dict(dtype="fp16", lens=[333, 64, 1], heads=40, kv=2, dim=128, page=16, group_size=64),  # twenty: two head tiles
    dict(dtype="bf16", lens=[333, 2500], heads=71, kv=1, dim=64, page=16),
    dict(dtype="fp16", lens=[513, 31], heads=8, kv=2, dim=256, page=16),
    dict(dtype="bf16", lens=[513, 2048], heads=24, kv=2, dim=256, page=128, group_size=64),
    dict(dtype="fp16", lens=[2048, 90], heads=14, kv=2, dim=256, page=48, group_size=128),
    dict(dtype="fp16", lens=[100, 5000], heads=8, kv=8, dim=128, page=1),
    dict(dtype="bf16", lens=[100, 5000, 640], heads=8, kv=2, dim=128, page=7, window=1),
    dict(dtype="fp16", lens=[100, 5000, 640, 0, 17], heads=8, kv=2, dim=128, page=17, window=17),
    dict(dtype="bf16", lens=[100, 5000, 640], heads=8, kv=2, dim=64, page=16, window=640),
    dict(dtype="fp16", lens=[65, 700], heads=8, kv=4, dim=128, page=16, q_pad=64, o_pad=8, page_pad=48),
    dict(dtype="fp16", lens=[3 * i % 97 for i in range(300)], heads=4, kv=2, dim=64, page=16),
    dict(dtype="bf16", lens=[7 * i % 41 for i in range(4096)], heads=2, kv=1, dim=64, page=16),  # the largest batch
    dict(dtype="fp16", lens=[66000, 3, 65536], heads=4, kv=1, dim=64, page=65536),  # the largest pages
    dict(dtype="bf16", lens=[66000, 3, 65535], heads=4, kv=1, dim=128, page=65535, window=600),
    dict(dtype="bf16", lens=[900, 40], heads=8, kv=2, dim=128, page=16, sigma=8.0),  # sharp softmax
    dict(dtype="fp16", lens=[3000, 40], heads=8, kv=2, dim=128, page=16, offset=3.0),  # values of one sign
    dict(dtype="bf16", lens=[700, 40], heads=8, kv=2, dim=128, page=16, group_size=64, q_sigma=2.0 ** 60, sigma=2.0 ** -60),
    dict(dtype="fp16", lens=[700, 40], heads=8, kv=2, dim=128, page=16, q_sigma=2.0 ** -9, sigma=512.0),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda c: f"{c['dtype']}h{c['heads']}kv{c['kv']}d{c['dim']}g{c.get('group_size', -1)}"
                         f"p{c['page']}w{c.get('window', 0)}n{max(c['lens'])}b{len(c['lens'])}")
def test_matches_formula(w4, kw):
    case = Case(w4, 11, **kw)
    ws = case.workspace()
    case.run(ws)
    case.check()
    assert w4.w4a16_status(ws) == 0


def test_repeats_and_changing_sizes_in_one_workspace(w4):
    """Every call gives the bits that it gives in a zeroed workspace of its own."""
    import torch
    cases = [Case(w4, 12, "fp16", [6000, 11, 350], 32, 8, 128, 16), Case(w4, 13, "bf16", [40, 9000, 0], 32, 8, 128, 16, 64),
             Case(w4, 14, "bf16", [53 * i % 300 for i in range(700)], 8, 4, 64, 16), Case(w4, 15, "fp16", [30000], 8, 1, 64, 64),
             Case(w4, 16, "fp16", [5000, 17], 8, 2, 256, 16), Case(w4, 17, "bf16", [20000, 9], 16, 1, 128, 64, window=15000)]
    alone = []
    for case in cases:
        case.run(case.workspace())
        case.check()
        alone.append((case.out.clone(), case.lse.clone()))
    shared = max((case.workspace() for case in cases), key=lambda ws: ws.numel())
    for i in (0, 2, 1, 3, 0, 4, 5, 2, 3, 3, 1, 4, 0, 5):
        case = cases[i]
        for x in (case.out, case.lse):
            x.fill_(float("nan"))
        case.run(shared)
        torch.cuda.synchronize()
        assert torch.equal(case.out, alone[i][0]) and torch.equal(case.lse, alone[i][1]), i
    assert w4.w4a16_status(shared) == 0


def test_lengths_grow_between_replays_on_a_side_stream(w4):
    """Lengths are read on the device: a captured call serves the next token too."""
    import torch
    case = Case(w4, 18, "fp16", [500, 64], 8, 2, 128, 16)
    ws = case.workspace()
    full = case.lens_list
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            case.run(ws, lse=False, stream=side)
            case.run(ws, stream=side)
        for lens in ([1, 0], [64, 63], [499, 64], full):
            case.lens.copy_(torch.tensor(lens, dtype=torch.int32))
            case.lens_list = lens
            graph.replay()
            side.synchronize()
            case.check()


def test_bad_lengths_and_pages_are_reported(w4):
    import torch
    case = Case(w4, 19, "fp16", [100, 200, 50], 8, 2, 128, 16)
    ws = case.workspace()
    case.lens[2] = -5
    case.run(ws)
    torch.cuda.synchronize()
    assert w4.w4a16_status(ws) == w4.W4A16_DEV_LENGTH
    case.lens_list[2] = 0
    case.check()
    case.lens[2] = case.max_pages * 16 + 1  # clamped: pages that the table does not have are then asked for
    case.run(ws)
    assert w4.w4a16_status(ws) == w4.W4A16_DEV_LENGTH | w4.W4A16_DEV_PAGE
    case.lens[2] = 0
    case.table[0, 3] = case.n_pages  # positions 48..63 of sequence 0 are then masked
    case.table[1, 0] = -1
    case.run(ws)
    assert w4.w4a16_status(ws) == w4.W4A16_DEV_PAGE
    case.check(dead={(0, p) for p in range(48, 64)} | {(1, p) for p in range(16)})
    case.lens[0] = case.lens_list[0] = 16
    case.table[0, 0] = -1  # nothing is left of sequence 0
    case.run(ws)
    case.check(dead={(0, p) for p in range(16)} | {(1, p) for p in range(16)})


@pytest.mark.parametrize("side", [0, 1])
def test_a_group_of_nan_makes_nan_of_what_it_touches(w4, side):
    import torch
    case = Case(w4, 20, "fp16", [300, 20], 8, 2, 128, 16, 64)
    ws = case.workspace()
    case.run(ws)
    torch.cuda.synchronize()
    before = case.out.clone()
    x = torch.randn((1, 2, 128), device="cuda").half()
    y = x.clone()
    (x, y)[side][0, 1, 70] = float("inf")  # KV head 1, its second group
    w4.w4a16_kv4_append(None, x, y, None, None, 0.0, None, case.cache, None, None, case.slots[0][7:8].contiguous(), None, 1, 0,
                        2, 128, 0, (), 0, 16, case.n_pages, 64, 0)
    case.run(ws)
    torch.cuda.synchronize()
    assert torch.equal(case.out[1], before[1])
    nan = torch.isnan(case.out[0].view(2, 4, 2, 64))
    assert not bool(nan[0].any())
    if side == 0:
        assert bool(nan[1].all())
    else:
        assert bool(nan[1, :, 1].all()) and not bool(nan[1, :, 0].any())


def test_a_cache_past_32_bits(w4):
    """Pages of many layers in one allocation: the last pages begin past 2^32 bytes."""
    import torch
    case = Case(w4, 21, "bf16", [5000, 300], 16, 4, 128, 32, page_pad=32 * 2 ** 20)
    assert case.cache.numel() > 2 ** 32
    ws = case.workspace()
    case.run(ws)
    case.check()
    assert w4.w4a16_status(ws) == 0


@pytest.mark.parametrize("dtype,dim,group_size", [("fp16", 128, -1), ("bf16", 128, 64), ("fp16", 64, -1)])
def test_records_with_negative_steps(w4, dtype, dim, group_size):
    """Values may as well be coded from the largest down."""
    case = Case(w4, 22, dtype, [700, 33], 8, 2, dim, 16, group_size)
    record = w4.w4a16_kv4_record_bytes(16, dim, group_size)
    rec = case.cache[:, :2 * record].view(-1, 2, record)
    rec[..., :16 * dim] ^= 0xFF
    sb = rec[..., 16 * dim:16 * dim + 32 * kv4.groups_of(dim, group_size) * 4].contiguous().view(kv4.TYPES[dtype])
    sb[..., 1::2] = (sb[..., 1::2].double() + 15 * sb[..., ::2].double()).to(sb.dtype)
    sb[..., ::2] *= -1
    import torch
    rec[..., 16 * dim:16 * dim + sb.shape[-1] * 2] = sb.view(torch.uint8)
    ws = case.workspace()
    case.run(ws)
    case.check()
    assert w4.w4a16_status(ws) == 0


def test_both_caches_attentions_in_one_workspace(w4):
    """The bits of workspaces of their own, in any order."""
    import torch
    case = Case(w4, 23, "fp16", [9000, 40, 2500], 32, 4, 128, 16)
    k, v = (torch.randn((case.n_pages, 16, 4, 128), device="cuda").half() for _ in range(2))
    out = torch.empty((3, 32 * 128), device="cuda", dtype=torch.float16)

    def paged(ws):
        w4.w4a16_paged_attention(case.q, k, v, out, case.table, case.lens, ws, 3, 32, 4, 128, 16, case.n_pages,
                                 case.max_pages, case.scale)

    size = w4.w4a16_paged_attention_workspace_size(3, 32, 4, 128)
    case.run(case.workspace())
    paged(torch.zeros(size, dtype=torch.uint8, device="cuda"))
    want = case.out.clone(), out.clone()
    shared = torch.zeros(max(size, case.workspace().numel()), dtype=torch.uint8, device="cuda")
    for turn in (0, 1, 0, 0, 1, 1, 0, 1):
        case.out.zero_()
        out.zero_()
        paged(shared) if turn else case.run(shared)
        torch.cuda.synchronize()
        assert torch.equal((case.out, out)[turn], want[turn])
    assert w4.w4a16_status(shared) == 0


def test_calls_side_by_side(w4):
    """Two streams, a workspace each: the bits of calls by themselves, directly and from graphs."""
    import torch
    cases = [Case(w4, 24, "fp16", [9000, 70], 32, 8, 128, 16), Case(w4, 25, "bf16", [300, 8000, 12], 16, 4, 128, 32, 64)]
    spaces = [case.workspace() for case in cases]
    want = []
    for case, ws in zip(cases, spaces):
        case.run(ws)
        torch.cuda.synchronize()
        want.append((case.out.clone(), case.lse.clone()))
        case.out.zero_()
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    graphs = []
    for case, ws, stream in zip(cases, spaces, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(5):
                case.run(ws, stream=stream)
        graphs.append(graph)
    for _ in range(10):
        for case, ws, stream, graph in zip(cases, spaces, streams, graphs):
            with torch.cuda.stream(stream):
                case.run(ws, stream=stream)
                graph.replay()
    torch.cuda.synchronize()
    for case, (out, lse) in zip(cases, want):
        assert torch.equal(case.out, out) and torch.equal(case.lse, lse)
