"""w4a16_paged_attention against its formula in 64 bits.

Tolerance.  A score is an fp32 sum of head_dim exact products (the tensor core adds 16 at a time):
an error of at most (D / 16 + 4) 2^-23 scale sum |q k|, which is below 2^-16 for the inputs here
(unit normals, scale D^-1/2: scale sum |q k| <= 30).  p therefore carries a relative error of 2^-15 at
most, and its 16-bit value plus remainder 2^-17 (bf16).  Both pass to the output as at most twice
that times max |v|.  So |out - ref| <= u |ref| + 2^-13 max |v| with u = 2^-11 (fp16) or 2^-8 (bf16), and
|lse - ref| <= 2^-14 + 2^-22 |ref|.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

UNIT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def w4():
    import torch
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    import weight_only_int4_03_gb300 as w4
    return w4


class Case:
    """Sequences of the given lengths over shuffled pages; cache rows that no sequence owns hold NaN."""

    def __init__(self, seed, dtype, lens, heads, kv, dim, page, window=0, order="token", q_pad=0, o_pad=0,
                 table_pad=0, sigma=1.0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        dt = torch.float16 if dtype == "fp16" else torch.bfloat16
        self.__dict__.update(dtype=dtype, lens_list=list(lens), heads=heads, kv=kv, dim=dim, page=page,
                             window=window, batch=len(lens), scale=dim ** -0.5)
        need = [(n + page - 1) // page for n in lens]
        self.n_pages = sum(need) + 2
        self.max_pages = max(max(need), 1)
        order_of = torch.randperm(self.n_pages, generator=g, device="cuda").to(torch.int32)
        # Unused table entries hold numbers that must not be looked up.
        self.table = torch.full((self.batch, self.max_pages + table_pad), -12345, dtype=torch.int32, device="cuda")
        k = torch.full((self.n_pages, page, kv, dim), float("nan"), dtype=dt, device="cuda")
        v = torch.full((self.n_pages, page, kv, dim), float("nan"), dtype=dt, device="cuda")
        self.dense = []
        at = 0
        for i, n in enumerate(lens):
            self.table[i, :need[i]] = order_of[at:at + need[i]]
            kk = torch.randn((n, kv, dim), generator=g, device="cuda", dtype=dt) * sigma
            vv = torch.randn((n, kv, dim), generator=g, device="cuda", dtype=dt)
            for j in range(need[i]):
                m = min(page, n - j * page)
                k[order_of[at + j], :m] = kk[j * page:j * page + m]
                v[order_of[at + j], :m] = vv[j * page:j * page + m]
            self.dense.append((kk, vv))
            at += need[i]
        self.strides = None
        if order == "head":  # [page][head][token][dim]
            k, v = k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous()
            self.strides = (kv * page * dim, dim, page * dim)
        self.k, self.v = k, v
        self.q = torch.randn((self.batch, heads * dim + q_pad), generator=g, device="cuda", dtype=dt)
        self.out = torch.full((self.batch, heads * dim + o_pad), float("nan"), device="cuda", dtype=dt)
        self.lse = torch.full((self.batch, heads), float("nan"), device="cuda")
        self.lens = torch.tensor(self.lens_list, dtype=torch.int32, device="cuda")

    def workspace(self, w4):
        import torch
        size = w4.w4a16_paged_attention_workspace_size(self.batch, self.heads, self.kv, self.dim)
        assert size > 0
        return torch.zeros(size, dtype=torch.uint8, device="cuda")

    def run(self, w4, ws, lse=True, **kw):
        w4.w4a16_paged_attention(self.q, self.k, self.v, self.out, self.table, self.lens, ws, self.batch,
                                 self.heads, self.kv, self.dim, self.page, self.n_pages, self.max_pages,
                                 self.scale, w4.W4A16_FLAG_BF16 if self.dtype == "bf16" else 0,
                                 window=self.window, lse=self.lse if lse else None, ldq=self.q.shape[1],
                                 ldo=self.out.shape[1], ld_table=self.table.shape[1], kv_strides=self.strides, **kw)

    def check(self):
        import torch
        torch.cuda.synchronize()
        group = self.heads // self.kv
        for i, n in enumerate(self.lens_list):
            got = self.out[i, :self.heads * self.dim].view(self.heads, self.dim).double()
            if n == 0:
                assert bool((got == 0).all())
                assert bool((self.lse[i] == float("-inf")).all())
                continue
            first = max(0, n - self.window) if self.window else 0
            k, v = (x[first:].double() for x in self.dense[i])
            q = self.q[i, :self.heads * self.dim].view(self.kv, group, self.dim).double()
            logits = torch.einsum("cgd,ncd->cgn", q, k) * self.scale
            ref = torch.einsum("cgn,ncd->cgd", torch.softmax(logits, -1), v).reshape(self.heads, self.dim)
            lse = torch.logsumexp(logits, -1).reshape(self.heads)
            tol = UNIT[self.dtype] * ref.abs() + 2.0 ** -13 * v.abs().max()
            err = (got - ref).abs()
            assert bool((err <= tol).all()), f"sequence {i} (length {n}): {float((err - tol).max())} over"
            assert bool(((self.lse[i].double() - lse).abs() <= 2.0 ** -14 + 2.0 ** -22 * lse.abs()).all()), i


CASES = [
    dict(dtype="fp16", lens=[1], heads=8, kv=2, dim=128, page=16),
    dict(dtype="bf16", lens=[37], heads=4, kv=4, dim=64, page=16),
    dict(dtype="fp16", lens=[0, 1, 15, 16, 17, 63, 64, 65, 0, 129], heads=16, kv=2, dim=128, page=16),
    dict(dtype="bf16", lens=[5, 300, 0, 2, 777], heads=12, kv=12, dim=64, page=24, table_pad=3),
    dict(dtype="fp16", lens=[4000], heads=5, kv=1, dim=128, page=64),
    dict(dtype="bf16", lens=[9001, 3], heads=40, kv=8, dim=128, page=32),
    dict(dtype="bf16", lens=[70, 1200], heads=9, kv=1, dim=128, page=8),         # nine heads: two row halves
    dict(dtype="fp16", lens=[70, 1200], heads=32, kv=2, dim=64, page=8),         # sixteen
    dict(dtype="fp16", lens=[333, 64, 1], heads=40, kv=2, dim=128, page=16),     # twenty: two head tiles
    dict(dtype="bf16", lens=[333, 2500], heads=71, kv=1, dim=64, page=16),
    dict(dtype="fp16", lens=[513, 31], heads=8, kv=2, dim=256, page=16),
    dict(dtype="bf16", lens=[513, 2048], heads=24, kv=2, dim=256, page=128),
    dict(dtype="fp16", lens=[100, 5000], heads=8, kv=8, dim=128, page=1),
    dict(dtype="bf16", lens=[100, 5000, 640], heads=8, kv=2, dim=128, page=7, window=1),
    dict(dtype="fp16", lens=[100, 5000, 640, 0, 17], heads=8, kv=2, dim=128, page=16, window=17),
    dict(dtype="bf16", lens=[100, 5000, 640], heads=8, kv=2, dim=64, page=16, window=640),
    dict(dtype="fp16", lens=[65, 700], heads=8, kv=4, dim=128, page=16, order="head", q_pad=64, o_pad=8),
    dict(dtype="fp16", lens=[3 * i % 97 for i in range(300)], heads=4, kv=2, dim=64, page=16),
    dict(dtype="bf16", lens=[900, 40], heads=8, kv=2, dim=128, page=16, sigma=8.0),  # sharp softmax
]


@pytest.mark.parametrize("kw", CASES, ids=lambda c: f"{c['dtype']}h{c['heads']}kv{c['kv']}d{c['dim']}"
                         f"p{c['page']}w{c.get('window', 0)}n{max(c['lens'])}b{len(c['lens'])}")
def test_matches_formula(w4, kw):
    if kw.get("sigma", 1.0) != 1.0:  # scores sigma times as large: their error bound too
        kw = dict(kw)
    case = Case(11, **kw)
    ws = case.workspace(w4)
    case.run(w4, ws)
    case.check()
    assert w4.w4a16_status(ws) == 0


def test_repeats_are_bit_identical_and_workspace_is_reusable(w4):
    import torch
    a = Case(12, "fp16", [6000, 11, 350], 32, 8, 128, 16)
    b = Case(13, "fp16", [40, 9000, 0], 32, 8, 128, 16)
    ws = a.workspace(w4)
    a.run(w4, ws)
    first, lse = a.out.clone(), a.lse.clone()
    for _ in range(5):
        b.run(w4, ws)
        a.run(w4, ws)
    torch.cuda.synchronize()
    assert torch.equal(a.out, first) and torch.equal(a.lse, lse)
    a.check()
    b.check()


def test_side_stream_graph_and_no_lse(w4):
    import torch
    case = Case(14, "bf16", [1000, 2, 77], 16, 4, 128, 16)
    ws = case.workspace(w4)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            case.run(w4, ws, lse=False, stream=side)
            case.run(w4, ws, lse=True, stream=side)
        graph.replay()
    side.synchronize()
    case.check()


def test_lengths_can_grow_between_replays(w4):
    """Lengths are read on the device: a captured call serves the next token too."""
    import torch
    case = Case(15, "fp16", [500, 64], 8, 2, 128, 16)
    ws = case.workspace(w4)
    full = case.lens_list
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        case.run(w4, ws)
    for lens in ([1, 0], [64, 63], [499, 64], full):
        case.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        keep = case.dense
        case.dense = [(k[:n], v[:n]) for (k, v), n in zip(keep, lens)]
        case.lens_list = lens
        graph.replay()
        case.check()
        case.dense = keep


def test_bad_lengths_and_pages_are_reported(w4):
    import torch
    case = Case(16, "fp16", [100, 200, 50], 8, 2, 128, 16)
    ws = case.workspace(w4)
    case.lens[2] = -5
    case.run(w4, ws)
    torch.cuda.synchronize()
    assert w4.w4a16_status(ws) == w4.W4A16_DEV_LENGTH
    case.lens_list[2] = 0
    case.check()
    case.lens[2] = 0
    case.table[0, 3] = case.n_pages  # positions 48..63 of sequence 0 are then masked
    case.run(w4, ws)
    torch.cuda.synchronize()
    assert w4.w4a16_status(ws) == w4.W4A16_DEV_PAGE
    k, v = case.dense[0]
    case.dense[0] = (torch.cat([k[:48], k[64:]]), torch.cat([v[:48], v[64:]]))
    case.lens_list[0] = 84
    case.check()


def test_offsets_past_32_bits(w4):
    """Pages more than 2^31 elements into the cache."""
    import torch
    if torch.cuda.get_device_properties(0).total_memory < 40 * 2 ** 30:
        pytest.skip("needs 20 GB")
    case = Case(17, "fp16", [200, 33], 4, 2, 128, 16)
    elems = 16 * 2 * 128
    n_pages = (2 ** 31 // elems) + 40
    k = torch.empty((n_pages, 16, 2, 128), dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    shift = n_pages - case.n_pages
    k[shift:] = case.k
    v[shift:] = case.v
    case.table[case.table >= 0] += shift
    case.k, case.v, case.n_pages = k, v, n_pages
    ws = case.workspace(w4)
    case.run(w4, ws)
    case.check()
    assert w4.w4a16_status(ws) == 0


@pytest.mark.parametrize("kw", [
    dict(dtype="fp16", lens=[1024], heads=4, kv=1, dim=128, page=16),          # 16 parts on 152 SMs: joined at once
    dict(dtype="bf16", lens=[1088], heads=8, kv=1, dim=128, page=16),          # 17: a group of 16 and one part
    dict(dtype="fp16", lens=[1100, 3], heads=16, kv=1, dim=64, page=24),       # 18, shared with a further row
    dict(dtype="bf16", lens=[2112, 0, 64, 1500], heads=12, kv=1, dim=256, page=64),
    dict(dtype="fp16", lens=[30000], heads=8, kv=1, dim=256, page=32),         # as many parts as blocks
    dict(dtype="bf16", lens=[30001, 17000], heads=20, kv=1, dim=128, page=16),
    dict(dtype="fp16", lens=[41000], heads=3, kv=1, dim=64, page=128),
    dict(dtype="bf16", lens=[9000, 70, 20000], heads=16, kv=2, dim=64, page=16, window=9001),
], ids=lambda c: f"{c['dtype']}h{c['heads']}d{c['dim']}n{max(c['lens'])}b{len(c['lens'])}")
def test_rows_in_many_parts(w4, kw):
    import torch
    case = Case(17, **kw)
    ws = case.workspace(w4)
    case.run(w4, ws)
    case.check()
    first, lse = case.out.clone(), case.lse.clone()
    for _ in range(3):
        case.run(w4, ws)
    torch.cuda.synchronize()
    assert torch.equal(case.out, first) and torch.equal(case.lse, lse)
    assert w4.w4a16_status(ws) == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("dim,heads,kv,batch", [(64, 8, 4, 120), (64, 64, 4, 120), (128, 8, 4, 80), (128, 48, 4, 80),
                                                (256, 8, 4, 40), (256, 64, 4, 40)])
@pytest.mark.parametrize("gap", [12.0, 17.4, 21.0])
def test_a_long_tail_under_dominant_positions_counts(w4, dtype, dim, heads, kv, batch, gap):
    """A few keys `gap` above thousands of equal ones whose values carry the output: the tail's p, 2^-17 to
    2^-30, is held as in l.

    Tolerance: the scores are single products, so p is off by 2^-20 of itself at most (the score's rounding in
    base 2 at 30, and exp2), plus 2^-17 (bf16's two parts), or 2^-23 and an absolute 2^-40 (fp16's): together
    below 2^-16 of the output and, fp16, 2^-40 / p.  Sums of equal signs and their join: 2^-13 at most (the
    MMA cuts off at 2^-23 of the sum, 16 positions at a time).  Then the last rounding.
    """
    import torch
    g = torch.Generator(device="cuda").manual_seed(18)
    dt = torch.float16 if dtype == "fp16" else torch.bfloat16
    n, page, scale = 2500, 128, dim ** -0.5
    pages = -(-n // page)
    dense = lambda: torch.randn((batch, n, kv, dim), generator=g, device="cuda", dtype=dt)
    k, v = dense(), dense().abs_().add_(1).mul_(8192)
    q = torch.zeros((batch, heads, dim), dtype=dt, device="cuda")
    q[:, :, 0] = 16
    k[..., 0] = 0
    k[:, :64:16, :, 0] = gap / (16 * scale)  # one in the first sixteen positions of every warp
    v[:, :64:16] = 0
    pad = lambda x: torch.cat([x, torch.full_like(x[:, :pages * page - n], float("nan"))], 1).view(-1, page, kv, dim)
    out, lse = torch.empty_like(q), torch.empty((batch, heads), device="cuda")
    table = torch.arange(batch * pages, device="cuda", dtype=torch.int32).view(batch, pages)
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    ws = torch.zeros(w4.w4a16_paged_attention_workspace_size(batch, heads, kv, dim), dtype=torch.uint8, device="cuda")
    w4.w4a16_paged_attention(q, pad(k), pad(v), out, table, lens, ws, batch, heads, kv, dim, page, batch * pages, pages,
                             scale, w4.W4A16_FLAG_BF16 if dtype == "bf16" else 0, lse=lse)
    torch.cuda.synchronize()
    logits = k[..., 0].double() * 16 * scale  # [batch, n, kv]
    p = torch.exp(logits - logits.amax(1, keepdim=True))
    ref = torch.einsum("bnc,bncd->bcd", p, v.double()) / p.sum(1)[..., None]
    ref = ref.repeat_interleave(heads // kv, 1)
    err = ((out.double() - ref).abs() / ref).max()
    tol = UNIT[dtype] + 2.0 ** -16 + 2.0 ** -13 + (2.0 ** -40 / float(p.min()) if dtype == "fp16" else 0.0)
    subnormal = 2.0 ** -25 / float(ref.min()) if dtype == "fp16" else 0.0
    assert float(err) <= tol + subnormal, (float(err), tol)
    want = torch.logsumexp(logits, 1).repeat_interleave(heads // kv, 1)
    assert bool(((lse.double() - want).abs() <= 2.0 ** -14 + 2.0 ** -22 * want.abs()).all())


@pytest.mark.parametrize("kw", [
    dict(dtype="fp16", lens=[7 * i % 130 for i in range(4096)], heads=4, kv=1, dim=64, page=16),
    dict(dtype="bf16", lens=[3000] + [1 + i % 40 for i in range(1200)] + [2000], heads=8, kv=2, dim=128, page=32),
], ids=("4096_short", "1202_between_long"))
def test_large_batches(w4, kw):
    case = Case(19, **kw)
    ws = case.workspace(w4)
    case.run(w4, ws)
    case.check()
    assert w4.w4a16_status(ws) == 0
