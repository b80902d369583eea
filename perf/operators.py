"""What the operators of a decode step around the W4A16 product are measured on.

Three operators: `rope` (rotary positions with one or several axes on q and k, k and v written
into a paged cache), `attention` (one new token per sequence over that cache) and `moe` (a whole
expert layer with 4-bit weights for a few tokens: router, top-k, gated products, down products,
weighted sum).  `run` computes them in elementary torch operations in fp32, or, where `own` is
true, through this package's entry points on the same state; `exact` computes them in fp64 from
the definition.
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# --- the cases -------------------------------------------------------------------------------

def listed():
    return [
        # A chat's first answered tokens, one user: nothing but latency.
        dict(name="attention_one_short", op="attention", dtype="fp16", batch=1, kv=8, group=4, dim=128,
             page=16, lo=37, hi=37, window=0),
        # One user deep into a long document: all of the card on one sequence.
        dict(name="attention_one_long", op="attention", dtype="bf16", batch=1, kv=8, group=5, dim=128,
             page=64, lo=131071, hi=131071, window=0),
        # A mixed batch of short and long chats, narrow heads without sharing, a sliding window.
        dict(name="attention_ragged_window", op="attention", dtype="fp16", batch=24, kv=12, group=1,
             dim=64, page=24, lo=5, hi=9000, window=2048),
        # A full server: ragged long sequences, grouped heads.
        dict(name="attention_server", op="attention", dtype="bf16", batch=32, kv=8, group=8, dim=128,
             page=32, lo=2048, hi=32768, window=0),
        # One new token of one user.
        dict(name="rope_one", op="rope", dtype="fp16", tokens=1, heads=32, kv=8, dim=128, rot=128,
             sections="64", adjacent=False, page=16),
        # A decode batch with narrow heads of which half are rotated, pairs side by side.
        dict(name="rope_batch_partial", op="rope", dtype="bf16", tokens=129, heads=16, kv=16, dim=64,
             rot=32, sections="16", adjacent=True, page=24),
        # A prefill of images and text: time, height and width positions.
        dict(name="rope_prefill_axes", op="rope", dtype="bf16", tokens=8191, heads=32, kv=8, dim=128,
             rot=128, sections="16,24,24", adjacent=False, page=64),
        # One token through a small layer of few experts.
        dict(name="moe_one_small", op="moe", dtype="fp16", tokens=1, hidden=1024, inter=1792, experts=8,
             top=2, group_size=128, zeros=False, act="silu", renorm=True),
        # One token through the framework's expert configuration (8 experts, 4096 x 14336, two each).
        dict(name="moe_one", op="moe", dtype="fp16", tokens=1, hidden=4096, inter=14336, experts=8, top=2,
             group_size=128, zeros=False, act="silu", renorm=True),
        # A few users on many narrow experts.
        dict(name="moe_many_experts", op="moe", dtype="bf16", tokens=7, hidden=2048, inter=768, experts=128,
             top=8, group_size=128, zeros=False, act="silu", renorm=True),
        # A decode batch on the same configuration with zero points: every expert is read.
        dict(name="moe_batch", op="moe", dtype="fp16", tokens=16, hidden=4096, inter=14336, experts=8, top=2,
             group_size=128, zeros=True, act="silu", renorm=True),
        # The widest call the layer takes, the other activation, weights not renormalised.
        dict(name="moe_widest", op="moe", dtype="bf16", tokens=64, hidden=4096, inter=14336, experts=8, top=2,
             group_size=64, zeros=False, act="gelu", renorm=False),
    ]


ATTENTION_MOST = 32 * 32768 * 8 * 128  # cached values of one side at the longest length
MOE_MOST = 8 * 4096 * 14336            # weights of one projection over all experts


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "rope", "moe", "moe"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "attention":
        dim = rng.choice([64, 128, 128, 256])
        kv = rng.choice([1, 2, 4, 8, 8, 12])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 20])
        if kv * group > 96:
            group = 8
        batch = _log_int(rng, 1, 64)
        longest = min(131072, ATTENTION_MOST // (batch * kv * dim))
        hi = _log_int(rng, 1, longest)
        lo = _log_int(rng, 1, hi)
        window = rng.choice([0, 0, 0, _log_int(rng, 1, hi)])
        return dict(op=op, dtype=dtype, batch=batch, kv=kv, group=group, dim=dim,
                    page=rng.choice([8, 16, 16, 24, 32, 64, 128]), lo=lo, hi=hi, window=window)
    if op == "rope":
        dim = rng.choice([64, 96, 128, 128, 256])
        rot = rng.choice([dim, dim, dim // 2])
        half = rot // 2
        cut = sorted(rng.sample(range(1, half), 2))
        sections = rng.choice([[half], [half], [cut[0], half - cut[0]],
                               [cut[0], cut[1] - cut[0], half - cut[1]]])
        kv = rng.choice([1, 2, 4, 8, 16])
        return dict(op=op, dtype=dtype, tokens=_log_int(rng, 1, 8191), heads=kv * rng.choice([1, 2, 4]),
                    kv=kv, dim=dim, rot=rot, sections=",".join(str(s) for s in sections),
                    adjacent=rng.choice([False, False, True]), page=rng.choice([8, 16, 24, 32, 64, 128]))
    experts = rng.choice([4, 8, 8, 16, 60, 64, 128])
    hidden = rng.choice([512, 768, 1024, 1280, 1536, 2048, 2560, 4096, 5120, 7168])
    inter = rng.choice([i for i in (256, 384, 512, 640, 768, 896, 1024, 1408, 1536, 1792, 2048, 2816, 3584, 4864,
                                    7168, 8192, 11008, 14336) if experts * hidden * i <= MOE_MOST])
    top = rng.choice([1, 2, 2, 4, 6, 8])
    group_size = rng.choice([64, 128, 128, -1])
    return dict(op="moe", dtype=dtype, tokens=_log_int(rng, 1, 64), hidden=hidden, inter=inter,
                experts=experts, top=min(top, experts), group_size=group_size,
                zeros=rng.choice([False, False, True]), act=rng.choice(["silu", "silu", "gelu"]),
                renorm=rng.choice([True, True, False]))


def lengths(case):
    """The sequences' lengths: spread over [lo, hi] in their logarithm, the longest first."""
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    out = []
    for i in range(n):
        f = 1.0 if i == 0 else (i * 0.6180339887498949) % 1.0
        out.append(max(lo, min(hi, int(round(lo * (hi / lo) ** f)))))
    return out


# --- the inputs ------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, sigma=1.0):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=dtype).mul_(sigma)


def _rand_int(g, lo, hi, shape, dtype=torch.int32):
    return torch.randint(lo, hi, shape, generator=g, device=DEVICE, dtype=dtype)


def _attention_state(case, seed):
    g = _generator(seed)
    dt = TYPES[case["dtype"]]
    b, kv, group, dim, page = case["batch"], case["kv"], case["group"], case["dim"], case["page"]
    lens = lengths(case)
    pages = [(n + page - 1) // page for n in lens]
    n_pages = sum(pages) + 3
    # Pages are handed out in any order, as a server's free list does after some time.
    order = torch.randperm(n_pages, generator=g, device=DEVICE).to(torch.int32)
    table = torch.zeros((b, max(pages)), dtype=torch.int32, device=DEVICE)
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = order[at:at + n]
        at += n
    s = dict(case=case, q=_randn(g, (b, kv * group, dim), dt),
             k_cache=_randn(g, (n_pages, page, kv, dim), dt),
             v_cache=_randn(g, (n_pages, page, kv, dim), dt), table=table,
             lens=torch.tensor(lens, dtype=torch.int32, device=DEVICE), scale=dim ** -0.5,
             out=torch.empty((b, kv * group, dim), dtype=dt, device=DEVICE),
             lse=torch.empty((b, kv * group), dtype=torch.float32, device=DEVICE))
    if own:
        import weight_only_int4_03_gb300 as w4
        s["flags"] = w4.W4A16_FLAG_BF16 if case["dtype"] == "bf16" else 0
        size = w4.w4a16_paged_attention_workspace_size(b, kv * group, kv, dim)
        s["workspace"] = torch.zeros(size, dtype=torch.uint8, device=DEVICE)
    return s


def _rope_state(case, seed):
    g = _generator(seed)
    dt = TYPES[case["dtype"]]
    t, heads, kv, dim, rot, page = (case[x] for x in ("tokens", "heads", "kv", "dim", "rot", "page"))
    sections = [int(x) for x in case["sections"].split(",")]
    max_pos = 32768
    n_pages = (t + page - 1) // page + 3
    # Frequencies theta^(-2i/rot) and the table of their angles, made once per model.
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEVICE) / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device=DEVICE)[:, None] * freq[None, :]
    table = torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()
    # One projection's output holds a token's q, k and v side by side.
    qkv = _randn(g, (t, (heads + 2 * kv) * dim), dt)
    slots = torch.randperm(n_pages * page, generator=g, device=DEVICE)[:t].contiguous()
    s = dict(case=case, qkv=qkv, table=table, sections=sections,
             positions=_rand_int(g, 0, max_pos, (len(sections), t)), slots=slots,
             k_cache=_randn(g, (n_pages, page, kv, dim), dt),
             v_cache=_randn(g, (n_pages, page, kv, dim), dt),
             q_out=torch.empty((t, heads, dim), dtype=dt, device=DEVICE))
    if own:
        import weight_only_int4_03_gb300 as w4
        s["flags"] = ((w4.W4A16_FLAG_BF16 if case["dtype"] == "bf16" else 0) |
                      (w4.W4A16_FLAG_ROPE_ADJACENT if case["adjacent"] else 0))
    return s


def _moe_weights(case, g, rows, cols):
    """One projection of every expert: packed codes [E][rows/8][cols], scales and zeros [E][G][cols]."""
    e, dt = case["experts"], TYPES[case["dtype"]]
    groups = 1 if case["group_size"] == -1 else rows // case["group_size"]
    words = _rand_int(g, -2 ** 31, 2 ** 31 - 1, (e, rows // 8, cols))
    scales = (torch.rand((e, groups, cols), generator=g, device=DEVICE) * 0.019 + 0.001).to(dt)
    zeros = _rand_int(g, 6, 10, (e, groups, cols)).to(dt) if case["zeros"] else None
    return words, scales, zeros


def _moe_state(case, seed):
    g = _generator(seed)
    dt = TYPES[case["dtype"]]
    t, h, i, e = case["tokens"], case["hidden"], case["inter"], case["experts"]
    x = _randn(g, (t, h), dt)
    router = _randn(g, (e, h), dt, 2.0 / math.sqrt(h))
    residual = _randn(g, (t, h), dt)
    up, up_s, up_z = _moe_weights(case, g, h, 2 * i)  # the I gate columns, then the I up columns
    down, down_s, down_z = _moe_weights(case, g, i, h)
    s = dict(case=case, x=x, router=router, residual=residual)
    if not own:
        s.update(up=up, up_s=up_s, up_z=up_z, down=down, down_s=down_s, down_z=down_z)
        return s
    import weight_only_int4_03_gb300 as w4

    def interleaved(src, rows):
        if src is None:
            return None
        dst = torch.empty_like(src)
        w4.w4_gate_up_interleave(src, dst, rows, 2 * i)
        return dst

    def packed(words, k, n):
        out = torch.empty((e, k * n // 8), dtype=torch.int32, device=DEVICE)
        for j in range(e):
            w4.w4_repack(words[j], None, out[j], k, n)
        return out

    groups = up_s.shape[1]
    flags = w4.W4A16_FLAG_SWIGLU if case["act"] == "silu" else w4.W4A16_FLAG_GEGLU
    if case["dtype"] == "bf16":
        flags |= w4.W4A16_FLAG_BF16
    if case["zeros"]:
        flags |= w4.W4A16_FLAG_HAS_ZP
    if case["renorm"]:
        flags |= w4.W4A16_FLAG_MOE_RENORM
    s.update(up=packed(interleaved(up, e * (h // 8)), h, 2 * i), up_s=interleaved(up_s, e * groups),
             up_z=interleaved(up_z, e * groups), down=packed(down, i, h), down_s=down_s, down_z=down_z,
             y=torch.empty((t, h), dtype=dt, device=DEVICE), flags=flags,
             weight_type=w4.W4A16_TYPE_U4 if case["zeros"] else w4.W4A16_TYPE_U4B8,
             workspace=torch.zeros(w4.w4a16_moe_layer_workspace_size(t, h, i, e, case["top"]),
                                   dtype=torch.uint8, device=DEVICE))
    torch.cuda.synchronize()  # the unpacked words go back to the allocator with this call's end
    return s


def prepare(case, seed):
    return {"attention": _attention_state, "rope": _rope_state, "moe": _moe_state}[case["op"]](case, seed)


# --- one pass --------------------------------------------------------------------------------

def _attention_plain(s):
    case = s["case"]
    b, kv, group, dim = case["batch"], case["kv"], case["group"], case["dim"]
    table = s["table"].long()
    k = s["k_cache"][table].flatten(1, 2).float()  # [b, positions, kv, dim]
    v = s["v_cache"][table].flatten(1, 2).float()
    q = s["q"].float().view(b, kv, group, dim)
    logits = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]  # [b, kv, group, positions]
    at = torch.arange(k.shape[1], device=DEVICE)[None, :]
    lens = s["lens"].long()[:, None]
    live = at < lens
    if case["window"]:
        live = live & (at >= lens - case["window"])
    logits = logits.masked_fill(~live[:, None, None, :], float("-inf"))
    top = logits.amax(dim=-1, keepdim=True)
    p = torch.exp(logits - top)
    total = p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p, v.permute(0, 2, 1, 3)) / total
    lse = (top + torch.log(total)).squeeze(-1)
    return out.view(b, kv * group, dim).to(s["q"].dtype), lse.view(b, kv * group)


def _attention_own(s):
    import weight_only_int4_03_gb300 as w4
    case = s["case"]
    w4.w4a16_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["out"], s["table"], s["lens"],
                             s["workspace"], case["batch"], case["kv"] * case["group"], case["kv"],
                             case["dim"], case["page"], s["k_cache"].shape[0], s["table"].shape[1],
                             s["scale"], s["flags"], window=case["window"], lse=s["lse"])
    return s["out"], s["lse"]


def _pair_axis(sections):
    return torch.tensor([a for a, n in enumerate(sections) for _ in range(n)], device=DEVICE)


def _rotate(x, cos, sin, rot, adjacent):
    """x [t, heads, dim]: the first `rot` values of every head are rotated in pairs."""
    y = x.clone()
    half = rot // 2
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if adjacent else (slice(0, half), slice(half, rot))
    a, b = x[..., first], x[..., second]
    c, s = cos[:, None, :], sin[:, None, :]
    y[..., first] = a * c - b * s
    y[..., second] = b * c + a * s
    return y


def _rope_plain(s):
    case = s["case"]
    t, heads, kv, dim, rot = (case[x] for x in ("tokens", "heads", "kv", "dim", "rot"))
    half = rot // 2
    dt = s["qkv"].dtype
    x = s["qkv"].float().view(t, heads + 2 * kv, dim)
    pair = torch.arange(half, device=DEVICE)
    at = s["positions"].long()[_pair_axis(s["sections"])].t()  # [t, half]
    cos, sin = s["table"][at, pair], s["table"][at, pair + half]
    turned = _rotate(x[:, :heads + kv], cos, sin, rot, case["adjacent"]).to(dt)
    s["k_cache"].view(-1, kv, dim)[s["slots"]] = turned[:, heads:]
    s["v_cache"].view(-1, kv, dim)[s["slots"]] = x[:, heads + kv:].to(dt)
    return turned[:, :heads].contiguous(), s["k_cache"], s["v_cache"]


def _rope_own(s):
    import weight_only_int4_03_gb300 as w4
    case = s["case"]
    heads, kv, dim = case["heads"], case["kv"], case["dim"]
    qkv = s["qkv"]
    ld = qkv.shape[1]
    w4.w4a16_rope_append(qkv, qkv[:, heads * dim:], qkv[:, (heads + kv) * dim:], s["q_out"], s["k_cache"],
                         s["v_cache"], s["table"], s["positions"], s["slots"], None, case["tokens"], heads,
                         kv, dim, case["rot"], s["sections"], s["table"].shape[0], case["page"],
                         s["k_cache"].shape[0], s["flags"], ldq=ld, ldk=ld, ldv=ld)
    return s["q_out"], s["k_cache"], s["v_cache"]


def _weights_plain(words, scales, zeros):
    """[..., K/8, N] words -> [..., K, N] fp32 weights (q - z) s, low nibble first."""
    shift = torch.arange(0, 32, 4, device=DEVICE, dtype=torch.int32)
    codes = ((words.unsqueeze(-2) >> shift[:, None]) & 15).flatten(-3, -2)  # [..., K, N]
    k = codes.shape[-2]
    groups = scales.shape[-2]
    w = codes.unflatten(-2, (groups, k // groups)).float()
    w = (w - (8.0 if zeros is None else zeros.float().unsqueeze(-2))) * scales.float().unsqueeze(-2)
    return w.flatten(-3, -2)


def _act_plain(x, act):
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))


def _route_plain(x, router, top, renorm):
    """The experts of each token, best first (the lowest index where scores are equal), and their weights."""
    logits = torch.matmul(x, router.t())
    p = torch.exp(logits - logits.amax(dim=-1, keepdim=True))
    p = p / p.sum(dim=-1, keepdim=True)
    order = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :top]
    w = p.gather(1, order)
    if renorm:
        w = w / w.sum(dim=-1, keepdim=True)
    return order, w


def _moe_plain(s):
    case = s["case"]
    t, inter, experts, top = case["tokens"], case["inter"], case["experts"], case["top"]
    x = s["x"].float()
    ids, weights = _route_plain(x, s["router"].float(), top, case["renorm"])
    y = s["residual"].float()

    def ffn(rows, pick):
        take = lambda v: None if v is None else (v[pick] if isinstance(pick, int) else v.index_select(0, pick)[0])
        gu = torch.matmul(rows, _weights_plain(take(s["up"]), take(s["up_s"]), take(s["up_z"])))
        h = _act_plain(gu[:, :inter], case["act"]) * gu[:, inter:]
        return torch.matmul(h, _weights_plain(take(s["down"]), take(s["down_s"]), take(s["down_z"])))

    if t * top < experts:  # the few experts that are asked for, read by index
        for a in range(t):
            for j in range(top):
                y[a:a + 1] += weights[a, j] * ffn(x[a:a + 1], ids[a, j:j + 1])
    else:  # every expert on every token, with weight 0 where it was not chosen
        full = torch.zeros((t, experts), device=DEVICE).scatter_(1, ids, weights)
        for e in range(experts):
            y += full[:, e:e + 1] * ffn(x, e)
    return y.to(s["x"].dtype)


def _moe_own(s):
    import weight_only_int4_03_gb300 as w4
    case = s["case"]
    w4.w4a16_moe_layer(s["x"], s["router"], s["up"], s["up_s"], s["up_z"], s["down"], s["down_s"], s["down_z"],
                       s["y"], s["workspace"], case["tokens"], case["hidden"], case["inter"], case["experts"],
                       case["top"], case["group_size"], s["weight_type"], s["flags"], residual=s["residual"])
    return s["y"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attention": _attention_own, "rope": _rope_own, "moe": _moe_own}[op](state)
    return {"attention": _attention_plain, "rope": _rope_plain, "moe": _moe_plain}[op](state)


# --- what a pass cannot do without -----------------------------------------------------------

def work(case):
    if case["op"] == "attention":
        lens = [min(n, case["window"]) if case["window"] else n for n in lengths(case)]
        rows = case["batch"] * case["kv"] * case["group"]
        pages = sum((n + case["page"] - 1) // case["page"] for n in lens)
        return {"bytes": sum(lens) * case["kv"] * case["dim"] * 4 + rows * (case["dim"] * 4 + 4) + 4 * pages +
                         4 * case["batch"],
                "flops": 4 * sum(lens) * case["kv"] * case["group"] * case["dim"]}
    if case["op"] == "rope":
        values = case["tokens"] * (case["heads"] + 2 * case["kv"]) * case["dim"]
        axes = len(case["sections"].split(","))
        table = case["tokens"] * case["rot"] * 4
        return {"bytes": values * 4 + table + case["tokens"] * (4 * axes + 8),
                "flops": 3 * case["tokens"] * (case["heads"] + case["kv"]) * case["rot"]}
    t, h, i, e, top = (case[x] for x in ("tokens", "hidden", "inter", "experts", "top"))
    active = max(top, round(e * (1.0 - (1.0 - top / e) ** t)))  # expected number of experts read
    per_group = 4 if case["zeros"] else 2
    up_groups = 1 if case["group_size"] == -1 else h // case["group_size"]
    down_groups = 1 if case["group_size"] == -1 else i // case["group_size"]
    expert = 3 * h * i // 2 + per_group * (up_groups * 2 * i + down_groups * h)
    return {"bytes": active * expert + 2 * e * h + 6 * t * h, "flops": 2 * t * e * h + 6 * t * top * h * i}


# --- the definition in 64 bits ---------------------------------------------------------------

def _attention_exact(case, s):
    b, kv, group, dim, page = case["batch"], case["kv"], case["group"], case["dim"], case["page"]
    out = torch.empty((b, kv * group, dim), dtype=torch.float64, device=DEVICE)
    lse = torch.empty((b, kv * group), dtype=torch.float64, device=DEVICE)
    for i, n in enumerate(lengths(case)):
        first = max(0, n - case["window"]) if case["window"] else 0
        at = torch.arange(first, n, device=DEVICE)
        rows = s["table"][i].long()[at // page] * page + at % page
        k = s["k_cache"].reshape(-1, kv, dim)[rows].double()
        v = s["v_cache"].reshape(-1, kv, dim)[rows].double()
        for c in range(kv):
            q = s["q"][i, c * group:(c + 1) * group].double()
            logits = (q @ k[:, c].t()) / math.sqrt(dim)
            out[i, c * group:(c + 1) * group] = torch.softmax(logits, dim=1) @ v[:, c]
            lse[i, c * group:(c + 1) * group] = torch.logsumexp(logits, dim=1)
    return out, lse


def _rope_exact(case, s):
    t, heads, kv, dim, rot = (case[x] for x in ("tokens", "heads", "kv", "dim", "rot"))
    half = rot // 2
    x = s["qkv"].double().view(t, heads + 2 * kv, dim)
    y = x.clone()
    i = 0
    for axis, count in enumerate(s["sections"]):
        rows = s["table"][s["positions"][axis].long()].double()
        for _ in range(count):
            c, n = rows[:, i, None], rows[:, half + i, None]
            p, r = (2 * i, 2 * i + 1) if case["adjacent"] else (i, half + i)
            y[:, :heads + kv, p] = x[:, :heads + kv, p] * c - x[:, :heads + kv, r] * n
            y[:, :heads + kv, r] = x[:, :heads + kv, p] * n + x[:, :heads + kv, r] * c
            i += 1
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    k_cache.view(-1, kv, dim)[s["slots"]] = y[:, heads:heads + kv]
    v_cache.view(-1, kv, dim)[s["slots"]] = y[:, heads + kv:]
    return y[:, :heads].contiguous(), k_cache, v_cache


def _expert_exact(words, scales, zeros, rows):
    """rows [t, K] in fp64 times one expert's weights, one nibble position of the words at a time."""
    k = words.shape[0] * 8
    group = k // scales.shape[0]
    total = None
    for i in range(8):
        at = torch.arange(i, k, 8, device=DEVICE)
        q = ((words >> (4 * i)) & 15).double()
        z = 8.0 if zeros is None else zeros.double()[at // group]
        part = rows[:, i::8] @ ((q - z) * scales.double()[at // group])
        total = part if total is None else total + part
    return total


def _moe_exact(case, s):
    inter, top = case["inter"], case["top"]
    x = s["x"].double()
    probability = torch.softmax(x @ s["router"].double().t(), dim=1).tolist()
    y = s["residual"].double()
    chosen = {}
    for t, row in enumerate(probability):
        best = sorted(range(len(row)), key=lambda e: (-row[e], e))[:top]
        total = sum(row[e] for e in best) if case["renorm"] else 1.0
        for e in best:
            chosen.setdefault(e, []).append((t, row[e] / total))
    for e, users in sorted(chosen.items()):
        at = torch.tensor([t for t, _ in users], device=DEVICE)
        w = torch.tensor([w for _, w in users], dtype=torch.float64, device=DEVICE)
        gu = _expert_exact(s["up"][e], s["up_s"][e], None if s["up_z"] is None else s["up_z"][e], x[at])
        g, u = gu[:, :inter], gu[:, inter:]
        if case["act"] == "silu":
            h = g * torch.sigmoid(g) * u
        else:
            h = g / 2 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3))) * u
        y.index_add_(0, at, w[:, None] * _expert_exact(
            s["down"][e], s["down_s"][e], None if s["down_z"] is None else s["down_z"][e], h))
    return y


def exact(case, seed):
    global own
    mine, own = own, False  # the inputs as a checkpoint holds them, whichever form is timed
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    return {"attention": _attention_exact, "rope": _rope_exact, "moe": _moe_exact}[case["op"]](case, s)
