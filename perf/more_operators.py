"""What the operators that complete a decode step are measured on.

Four operators: `norm_rope` (queries and keys normalised per head and rotated, keys and values written
into a paged cache of 16 bits), `kv4_append` (the same into a paged cache held in 4 bits), `kv4_attention`
(one new token per sequence over that cache) and `sample` (the next token of each row of logits, by
temperature, top-k, top-p and min-p, from given uniform numbers).  `run` computes them in elementary
torch operations, or, where `own` is true, through this package's entry points on the same inputs;
`exact` computes them in fp64 from the definition.

A group of values in 4 bits: b = min and s = (max - min) / 15, both rounded to the cache's 16-bit type, a code
q = (x - b) / s rounded to the nearest integer (ties to even) in 0..15, and q s + b the value it stands for.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# --- the cases -------------------------------------------------------------------------------

def listed():
    return [
        # A chat's first answered tokens, one user: nothing but latency.
        dict(name="kv4_attention_one_short", op="kv4_attention", dtype="fp16", batch=1, kv=8, group=4, dim=128,
             group_size=-1, page=16, lo=41, hi=41, window=0),
        # One user deep into a long document: all of the card on one sequence.
        dict(name="kv4_attention_one_long", op="kv4_attention", dtype="bf16", batch=1, kv=8, group=5, dim=128,
             group_size=64, page=64, lo=131071, hi=131071, window=0),
        # A mixed batch of short and long chats, narrow heads without sharing, a sliding window.
        dict(name="kv4_attention_ragged_window", op="kv4_attention", dtype="fp16", batch=24, kv=12, group=1, dim=64,
             group_size=-1, page=24, lo=5, hi=9000, window=2048),
        # A full server: ragged long sequences, grouped heads.
        dict(name="kv4_attention_server", op="kv4_attention", dtype="bf16", batch=48, kv=8, group=8, dim=128,
             group_size=-1, page=32, lo=2048, hi=32768, window=0),
        # One new token of one user.
        dict(name="kv4_append_one", op="kv4_append", dtype="fp16", tokens=1, heads=32, kv=8, dim=128, rot=128,
             sections="64", adjacent=False, norm=True, group_size=-1, page=16),
        # A prompt of text and images: time, height and width positions, groups of 64.
        dict(name="kv4_append_prefill_axes", op="kv4_append", dtype="bf16", tokens=8191, heads=32, kv=8, dim=128,
             rot=128, sections="16,24,24", adjacent=False, norm=True, group_size=64, page=64),
        # A decode batch into the cache of 16 bits, heads of 256 of which half is rotated, pairs side by side.
        dict(name="norm_rope_batch_partial", op="norm_rope", dtype="fp16", tokens=129, heads=16, kv=2, dim=256, rot=128,
             sections="64", adjacent=True, norm=True, page=24),
        # A prompt into the cache of 16 bits.
        dict(name="norm_rope_prefill", op="norm_rope", dtype="bf16", tokens=6007, heads=32, kv=8, dim=128, rot=128,
             sections="64", adjacent=False, norm=True, page=64),
        # One user's next token, plain settings of a chat.
        dict(name="sample_one", op="sample", dtype="fp16", batch=1, vocab=32000, sigma=3.0, kind="chat", masked=0.0),
        # A decode batch whose rows each have settings of their own, greedy ones among them.
        dict(name="sample_batch_mixed", op="sample", dtype="bf16", batch=48, vocab=131071, sigma=2.5, kind="mixed",
             masked=0.0),
        # Sampling without filters from a wide vocabulary.
        dict(name="sample_batch_open", op="sample", dtype="fp16", batch=32, vocab=256000, sigma=2.0, kind="open",
             masked=0.0),
        # A large batch under a grammar: most of the vocabulary is masked out.
        dict(name="sample_large_masked", op="sample", dtype="fp16", batch=256, vocab=100003, sigma=3.0, kind="mixed",
             masked=0.9),
    ]


ATTENTION_MOST = 480_000_000  # cached values of one side, were every sequence as long as the longest
SAMPLE_MOST = 256 * 100003             # logits


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_rotation(rng, dim):
    rot = rng.choice([dim, dim, dim // 2])
    half = rot // 2
    cut = sorted(rng.sample(range(1, half), 2))
    sections = rng.choice([[half], [half], [cut[0], half - cut[0]], [cut[0], cut[1] - cut[0], half - cut[1]]])
    return dict(rot=rot, sections=",".join(str(n) for n in sections), adjacent=rng.choice([False, False, True]),
                norm=rng.choice([True, True, False]))


def draw(rng):
    op = rng.choice(["kv4_attention", "kv4_attention", "kv4_append", "norm_rope", "sample", "sample"])
    dtype = rng.choice(["fp16", "bf16"])
    page = rng.choice([8, 16, 16, 24, 32, 64, 128])
    if op == "kv4_attention":
        dim = rng.choice([64, 128, 128, 256])
        kv = rng.choice([1, 2, 4, 8, 8, 12])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16, 20])
        if kv * group > 96:
            group = 8
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, min(131072, ATTENTION_MOST // (batch * kv * dim)))
        return dict(op=op, dtype=dtype, batch=batch, kv=kv, group=group, dim=dim,
                    group_size=rng.choice([-1, -1, 64, min(128, dim)]), page=page, lo=_log_int(rng, 1, hi), hi=hi,
                    window=rng.choice([0, 0, 0, _log_int(rng, 1, hi)]))
    if op == "sample":
        vocab = _log_int(rng, 1000, 262144)
        return dict(op=op, dtype=dtype, batch=_log_int(rng, 1, min(256, SAMPLE_MOST // vocab)), vocab=vocab,
                    sigma=round(rng.uniform(1.5, 5.0), 2), kind=rng.choice(["chat", "mixed", "mixed", "open"]),
                    masked=rng.choice([0.0, 0.0, 0.5, 0.99]))
    kv = rng.choice([1, 2, 4, 8])
    case = dict(op=op, dtype=dtype, tokens=_log_int(rng, 1, 6007), heads=kv * rng.choice([1, 2, 4]), kv=kv, page=page)
    if op == "kv4_append":
        dim = rng.choice([64, 128, 128, 256])
        return dict(case, dim=dim, group_size=rng.choice([-1, 64, min(128, dim)]), **_draw_rotation(rng, dim))
    dim = rng.choice([64, 96, 128, 128, 256])
    return dict(case, dim=dim, **_draw_rotation(rng, dim))


def lengths(case):
    """The sequences' lengths: spread over [lo, hi] in their logarithm, the longest first."""
    n, lo, hi = case["batch"], case["lo"], case["hi"]
    spread = [1.0] + [(i * 0.6180339887498949) % 1.0 for i in range(1, n)]
    return [max(lo, min(hi, int(round(lo * (hi / lo) ** f)))) for f in spread]


# --- the inputs ------------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _randn(g, shape, dtype, sigma=1.0):
    return torch.randn(shape, generator=g, device=DEVICE, dtype=dtype).mul_(sigma)


def _groups(case):
    return 1 if case["group_size"] == -1 else case["dim"] // case["group_size"]


def _quantise(x, groups, dtype):
    """x [..., dim] -> codes [..., groups, dim / groups] and (s, b) [..., groups] in the cache's type, in x's precision."""
    x = x.unflatten(-1, (groups, x.shape[-1] // groups))
    lo, hi = x.amin(-1), x.amax(-1)
    b, s = lo.to(dtype), ((hi - lo) / 15).to(dtype)
    step = s.to(x.dtype).unsqueeze(-1)
    codes = ((x - b.to(x.dtype).unsqueeze(-1)) / step).round().clamp(0, 15)
    return torch.where(step > 0, codes, torch.zeros_like(codes)), s, b


def _pack(codes):
    """[..., groups, values] codes -> [..., dim / 2] bytes, the first of two in the low half."""
    codes = codes.flatten(-2).to(torch.uint8)
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _flags(case):
    import weight_only_int4_03_gb300 as w4
    return ((w4.W4A16_FLAG_BF16 if case["dtype"] == "bf16" else 0) |
            (w4.W4A16_FLAG_ROPE_ADJACENT if case.get("adjacent") else 0))


def _kv4_cache(case, n_pages):
    import weight_only_int4_03_gb300 as w4
    record = w4.w4a16_kv4_record_bytes(case["page"], case["dim"], case["group_size"])
    return torch.zeros((n_pages, case["kv"] * record), dtype=torch.uint8, device=DEVICE)


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
    s = dict(case=case, q=_randn(g, (b, kv * group, dim), dt), table=table, pages=n_pages,
             lens=torch.tensor(lens, dtype=torch.int32, device=DEVICE), scale=dim ** -0.5)
    # Keys whose channels differ in size and offset, as trained ones do.
    size = torch.exp(_randn(g, (2, kv, dim), torch.float32, 0.3))
    offset = _randn(g, (kv, dim), torch.float32, 0.5)
    if own:
        import weight_only_int4_03_gb300 as w4
        s.update(flags=_flags(case), cache=_kv4_cache(case, n_pages),
                 out=torch.empty((b, kv * group, dim), dtype=dt, device=DEVICE),
                 lse=torch.empty((b, kv * group), dtype=torch.float32, device=DEVICE),
                 workspace=torch.zeros(w4.w4a16_kv4_attention_workspace_size(b, kv * group, kv, dim),
                                       dtype=torch.uint8, device=DEVICE))
    else:
        s["codes"] = torch.empty((2, n_pages, page, kv, dim // 2), dtype=torch.uint8, device=DEVICE)
        s["params"] = torch.empty((2, 2, n_pages, page, kv, _groups(case)), dtype=dt, device=DEVICE)
    chunk = max(1, 2 ** 26 // (page * kv * dim))
    for first in range(0, n_pages, chunk):
        n = min(chunk, n_pages - first)
        k = (_randn(g, (n, page, kv, dim), torch.float32) * size[0] + offset).to(dt)
        v = (_randn(g, (n, page, kv, dim), torch.float32) * size[1]).to(dt)
        if own:
            slots = torch.arange(first * page, (first + n) * page, device=DEVICE)
            w4.w4a16_kv4_append(None, k, v, None, None, 0.0, None, s["cache"], None, None, slots, None, n * page, 0,
                                kv, dim, 0, (), 0, page, n_pages, case["group_size"], s["flags"])
            continue
        for side, x in enumerate((k, v)):
            codes, step, base = _quantise(x.float(), _groups(case), dt)
            s["codes"][side, first:first + n] = _pack(codes)
            s["params"][side, 0, first:first + n] = step
            s["params"][side, 1, first:first + n] = base
    return s


def _append_state(case, seed):
    g = _generator(seed)
    dt = TYPES[case["dtype"]]
    t, heads, kv, dim, rot, page = (case[x] for x in ("tokens", "heads", "kv", "dim", "rot", "page"))
    sections = tuple(int(x) for x in case["sections"].split(","))
    max_pos = 32768
    n_pages = (t + page - 1) // page + 3
    # Frequencies theta^(-2i/rot) and the table of their angles, made once per model.
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEVICE) / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device=DEVICE)[:, None] * freq[None, :]
    table = torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous()
    # One projection's output holds a token's q, k and v side by side.
    s = dict(case=case, qkv=_randn(g, (t, (heads + 2 * kv) * dim), dt), table=table, sections=sections,
             positions=torch.randint(0, max_pos, (len(sections), t), generator=g, device=DEVICE, dtype=torch.int32),
             slots=torch.randperm(n_pages * page, generator=g, device=DEVICE)[:t].contiguous(),
             q_norm=None, k_norm=None, eps=1e-6, pages=n_pages)
    if case["norm"]:
        s["q_norm"], s["k_norm"] = (1.0 + 0.2 * _randn(g, (2, dim), torch.float32)).to(dt)
    if case["op"] == "norm_rope":
        s["k_cache"], s["v_cache"] = (_randn(g, (n_pages, page, kv, dim), dt) for _ in range(2))
    if own:
        s["flags"] = _flags(case)
        s["q_out"] = torch.empty((t, heads, dim), dtype=dt, device=DEVICE)
        if case["op"] == "kv4_append":
            s["cache"] = _kv4_cache(case, n_pages)
            s["k_out"], s["v_out"] = (torch.empty((t, kv, dim), dtype=dt, device=DEVICE) for _ in range(2))
    return s


def _sample_state(case, seed):
    g = _generator(seed)
    b, vocab = case["batch"], case["vocab"]
    # The product that makes the logits has its columns padded.
    padded = (vocab + 255) // 256 * 256
    logits = _randn(g, (b, padded), torch.float32, case["sigma"])
    if case["masked"]:
        allowed = torch.rand((b, padded), generator=g, device=DEVICE) >= case["masked"]
        logits = logits.masked_fill(~allowed, float("-inf"))
    s = dict(case=case, logits=logits.to(TYPES[case["dtype"]]),
             uniform=torch.rand(b, generator=g, device=DEVICE), temperature=None, top_k=None, top_p=None, min_p=None)

    def pick(values, dtype):
        at = torch.randint(0, len(values), (b,), generator=g, device=DEVICE)
        return torch.tensor(values, dtype=dtype, device=DEVICE)[at]

    if case["kind"] == "chat":
        s["temperature"], s["top_k"] = pick([0.7, 0.8], torch.float32), pick([40, 50], torch.int32)
        s["top_p"] = pick([0.95, 0.9], torch.float32)
    elif case["kind"] == "mixed":
        s["temperature"] = pick([0.0, 0.5, 0.7, 1.0, 1.0, 1.3], torch.float32)
        s["top_k"] = pick([0, 0, 1, 20, 50, 1000], torch.int32)
        s["top_p"] = pick([1.0, 1.0, 0.99, 0.95, 0.9, 0.5], torch.float32)
        s["min_p"] = pick([0.0, 0.0, 0.02, 0.1], torch.float32)
    if own:
        s["flags"] = _flags(case)
        s["tokens"] = torch.empty(b, dtype=torch.int32, device=DEVICE)
        s["logprobs"] = torch.empty(b, dtype=torch.float32, device=DEVICE)
    return s


def prepare(case, seed):
    return {"kv4_attention": _attention_state, "kv4_append": _append_state, "norm_rope": _append_state,
            "sample": _sample_state}[case["op"]](case, seed)


# --- one pass --------------------------------------------------------------------------------

def _values(s, side, table):
    """The cached values of one side that the tables name, [batch, positions, kv, dim] in fp32."""
    codes = s["codes"][side][table].flatten(1, 2)
    step, base = (s["params"][side, i][table].flatten(1, 2).float() for i in range(2))
    codes = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).unflatten(-1, (step.shape[-1], -1))
    return (codes * step.unsqueeze(-1) + base.unsqueeze(-1)).flatten(-2)


def _attention_plain(s):
    case = s["case"]
    b, kv, group, dim = case["batch"], case["kv"], case["group"], case["dim"]
    table = s["table"].long()
    k = _values(s, 0, table)
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
    out = torch.matmul(p, _values(s, 1, table).permute(0, 2, 1, 3)) / total
    lse = (top + torch.log(total)).squeeze(-1)
    return out.view(b, kv * group, dim).to(s["q"].dtype), lse.view(b, kv * group)


def _attention_own(s):
    import weight_only_int4_03_gb300 as w4
    case = s["case"]
    w4.w4a16_kv4_attention(s["q"], s["cache"], s["out"], s["table"], s["lens"], s["workspace"], case["batch"],
                           case["kv"] * case["group"], case["kv"], case["dim"], case["page"], s["pages"],
                           s["table"].shape[1], case["group_size"], s["scale"], s["flags"], window=case["window"],
                           lse=s["lse"])
    return s["out"], s["lse"]


def _turned(s, x, weight, precision):
    """x [tokens, heads, dim] of the projection: normalised per head, then rotated."""
    case = s["case"]
    rot = case["rot"]
    half = rot // 2
    x = x.to(precision)
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + s["eps"]) * weight.to(precision)
    sizes = torch.tensor(s["sections"], device=DEVICE)
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=DEVICE), sizes, output_size=half)
    pair = torch.arange(half, device=DEVICE)
    at = s["positions"].long()[axis].t()  # [tokens, half]
    c, n = (s["table"][at, pair + i * half].to(precision)[:, None, :] for i in range(2))
    first, second = ((slice(0, rot, 2), slice(1, rot, 2)) if case["adjacent"] else
                     (slice(0, half), slice(half, rot)))
    a, b = x[..., first], x[..., second]
    y = x.clone()
    y[..., first] = a * c - b * n
    y[..., second] = b * c + a * n
    return y


def _split(s):
    case = s["case"]
    x = s["qkv"].view(case["tokens"], case["heads"] + 2 * case["kv"], case["dim"])
    return x.split((case["heads"], case["kv"], case["kv"]), dim=1)


def _norm_rope_plain(s):
    dt = s["qkv"].dtype
    q, k, v = _split(s)
    s["k_cache"].flatten(0, 1)[s["slots"]] = _turned(s, k, s["k_norm"], torch.float32).to(dt)
    s["v_cache"].flatten(0, 1)[s["slots"]] = v
    return _turned(s, q, s["q_norm"], torch.float32).to(dt).contiguous(), s["k_cache"], s["v_cache"]


def _kv4_append_plain(s):
    dt, groups = s["qkv"].dtype, _groups(s["case"])
    q, k, v = _split(s)
    out = [_turned(s, q, s["q_norm"], torch.float32).to(dt).contiguous()]
    # In 64 bits: many values lie next to the border of two codes.
    for x in (_turned(s, k, s["k_norm"], torch.float64), v.double()):
        codes, step, base = _quantise(x, groups, dt)
        out.append((codes * step.unsqueeze(-1) + base.unsqueeze(-1)).flatten(-2).to(dt))
    return tuple(out)


def _parts_own(s):
    case = s["case"]
    heads, kv, dim = case["heads"], case["kv"], case["dim"]
    qkv = s["qkv"]
    ld = qkv.shape[1]
    return (qkv, qkv[:, heads * dim:], qkv[:, (heads + kv) * dim:]), dict(ldq=ld, ldk=ld, ldv=ld)


def _norm_rope_own(s):
    import weight_only_int4_03_gb300 as w4
    case = s["case"]
    parts, strides = _parts_own(s)
    w4.w4a16_norm_rope_append(*parts, s["q_norm"], s["k_norm"], s["eps"], s["q_out"], s["k_cache"], s["v_cache"],
                              s["table"], s["positions"], s["slots"], None, case["tokens"], case["heads"], case["kv"],
                              case["dim"], case["rot"], s["sections"], s["table"].shape[0], case["page"], s["pages"],
                              s["flags"], **strides)
    return s["q_out"], s["k_cache"], s["v_cache"]


def _kv4_append_own(s):
    import weight_only_int4_03_gb300 as w4
    case = s["case"]
    parts, strides = _parts_own(s)
    w4.w4a16_kv4_append(*parts, s["q_norm"], s["k_norm"], s["eps"], s["q_out"], s["cache"], s["table"],
                        s["positions"], s["slots"], None, case["tokens"], case["heads"], case["kv"], case["dim"],
                        case["rot"], s["sections"], s["table"].shape[0], case["page"], s["pages"],
                        case["group_size"], s["flags"], k_out=s["k_out"], v_out=s["v_out"], **strides)
    return s["q_out"], s["k_out"], s["v_out"]


def _setting(s, name, default, dtype):
    b = s["case"]["batch"]
    v = s[name]
    v = torch.full((b,), default, dtype=dtype, device=DEVICE) if v is None else v.to(dtype)
    return v[:, None]


def _sample_plain(s):
    # In 64 bits: the token is decided by where a number falls among sums of up to a whole vocabulary.
    vocab = s["case"]["vocab"]
    logits = s["logits"][:, :vocab].double()
    t = _setting(s, "temperature", 1.0, torch.float64)
    greedy = t == 0
    top = logits.amax(dim=1, keepdim=True)
    w = torch.exp((logits - top) / torch.where(greedy, torch.ones_like(t), t))
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices
    best = w.gather(1, order)
    rank = torch.arange(vocab, device=DEVICE)[None, :]
    k = _setting(s, "top_k", 0, torch.int64)
    best = torch.where((k <= 0) | (rank < k), best, torch.zeros_like(best))
    total = best.cumsum(1)
    p = _setting(s, "top_p", 1.0, torch.float64)
    keep = ((p >= 1) | (total - best < p * total[:, -1:]) | (rank == 0)) & (best > 0)
    keep = keep & (best >= _setting(s, "min_p", 0.0, torch.float64).clamp(max=1.0))
    w = w * torch.zeros_like(w).scatter_(1, order, keep.double())
    total = w.cumsum(1)
    token = (total <= s["uniform"].double()[:, None] * total[:, -1:]).sum(dim=1, keepdim=True)
    first = torch.where(logits == top, rank, vocab).amin(dim=1, keepdim=True)
    logprob = torch.log(w.gather(1, token.clamp(max=vocab - 1)) / total[:, -1:])
    token = torch.where(greedy, first, token)
    logprob = torch.where(greedy, torch.zeros_like(logprob), logprob)
    return token.squeeze(1).to(torch.int32), logprob.squeeze(1).float()


def _sample_own(s):
    import weight_only_int4_03_gb300 as w4
    case = s["case"]
    w4.w4a16_sample(s["logits"], s["uniform"], s["tokens"], case["batch"], case["vocab"], s["flags"],
                    temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"],
                    logprobs=s["logprobs"], ld=s["logits"].shape[1])
    return s["tokens"], s["logprobs"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"kv4_attention": _attention_own, "kv4_append": _kv4_append_own, "norm_rope": _norm_rope_own,
                "sample": _sample_own}[op](state)
    return {"kv4_attention": _attention_plain, "kv4_append": _kv4_append_plain, "norm_rope": _norm_rope_plain,
            "sample": _sample_plain}[op](state)


# --- what a pass cannot do without -----------------------------------------------------------

def work(case):
    if case["op"] == "kv4_attention":
        lens = [min(n, case["window"]) if case["window"] else n for n in lengths(case)]
        rows = case["batch"] * case["kv"] * case["group"]
        pages = sum((n + case["page"] - 1) // case["page"] for n in lens)
        return {"bytes": sum(lens) * case["kv"] * (case["dim"] + 8 * _groups(case)) + rows * (case["dim"] * 4 + 4) +
                         4 * pages + 4 * case["batch"],
                "flops": 4 * sum(lens) * case["kv"] * case["group"] * case["dim"]}
    if case["op"] == "sample":
        return {"bytes": case["batch"] * (2 * case["vocab"] + 28), "flops": 4 * case["batch"] * case["vocab"]}
    t, kv, dim = case["tokens"], case["kv"], case["dim"]
    read = t * (case["heads"] + 2 * kv) * dim * 2 + t * (case["rot"] * 4 + 4 * len(case["sections"].split(",")) + 8)
    written = t * (case["heads"] + 2 * kv) * dim * 2
    if case["op"] == "kv4_append":
        written += t * kv * (dim + 8 * _groups(case))
    return {"bytes": read + written + 4 * dim,
            "flops": t * (case["heads"] + kv) * (3 * case["rot"] + (4 * dim if case["norm"] else 0))}


# --- the definition in 64 bits ---------------------------------------------------------------

def _attention_exact(case, s):
    b, kv, group, dim, page = case["batch"], case["kv"], case["group"], case["dim"], case["page"]
    size = dim // _groups(case)
    out = torch.empty((b, kv * group, dim), dtype=torch.float64, device=DEVICE)
    lse = torch.empty((b, kv * group), dtype=torch.float64, device=DEVICE)
    for i, n in enumerate(lengths(case)):
        first = max(0, n - case["window"]) if case["window"] else 0
        at = torch.arange(first, n, device=DEVICE)
        pages, tokens = s["table"][i].long()[at // page], at % page
        for c in range(kv):
            sides = []
            for side in range(2):
                packed = s["codes"][side][pages, tokens, c]
                x = torch.empty((n - first, dim), dtype=torch.float64, device=DEVICE)
                x[:, 0::2], x[:, 1::2] = (packed % 16).double(), (packed // 16).double()
                step, base = (s["params"][side, j][pages, tokens, c].double().repeat_interleave(size, dim=1)
                              for j in range(2))
                sides.append(x * step + base)
            logits = (s["q"][i, c * group:(c + 1) * group].double() @ sides[0].t()) / math.sqrt(dim)
            out[i, c * group:(c + 1) * group] = torch.softmax(logits, dim=1) @ sides[1]
            lse[i, c * group:(c + 1) * group] = torch.logsumexp(logits, dim=1)
    return out, lse


def _turned_exact(case, s, x, weight):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["dim"] + s["eps"]) * weight.double()
    y, i, half = x.clone(), 0, case["rot"] // 2
    for axis, count in enumerate(s["sections"]):
        rows = s["table"][s["positions"][axis].long()].double()
        for _ in range(count):
            c, n = rows[:, i, None], rows[:, half + i, None]
            p, r = (2 * i, 2 * i + 1) if case["adjacent"] else (i, half + i)
            y[:, :, p] = x[:, :, p] * c - x[:, :, r] * n
            y[:, :, r] = x[:, :, p] * n + x[:, :, r] * c
            i += 1
    return y


def _append_exact(case, s):
    t, heads, kv, dim = case["tokens"], case["heads"], case["kv"], case["dim"]
    x = s["qkv"].view(t, heads + 2 * kv, dim)
    q = _turned_exact(case, s, x[:, :heads], s["q_norm"])
    k, v = _turned_exact(case, s, x[:, heads:heads + kv], s["k_norm"]), x[:, heads + kv:].double()
    if case["op"] == "norm_rope":
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        k_cache.view(-1, kv, dim)[s["slots"]] = k
        v_cache.view(-1, kv, dim)[s["slots"]] = v
        return q, k_cache, v_cache
    size = dim // _groups(case)
    dt = s["qkv"].dtype
    for x in (k, v):
        for at in range(0, dim, size):
            part = x[:, :, at:at + size]
            low, high = part.min(dim=-1, keepdim=True).values, part.max(dim=-1, keepdim=True).values
            step, base = ((high - low) / 15.0).to(dt).double(), low.to(dt).double()
            code = torch.round((part - base) / torch.where(step > 0, step, torch.ones_like(step)))
            part.copy_(base + step * torch.clamp(code, min=0.0, max=15.0))
    return q, k, v


def _sample_exact(case, s):
    def column(name, default):
        return [default] * case["batch"] if s[name] is None else s[name].tolist()

    rows = s["logits"][:, :case["vocab"]].double().cpu().numpy()
    tokens, logprobs = [], []
    for x, u, t, k, p, least in zip(rows, s["uniform"].tolist(), column("temperature", 1.0), column("top_k", 0),
                                    column("top_p", 1.0), column("min_p", 0.0)):
        if t == 0:
            tokens.append(int(np.argmax(x)))
            logprobs.append(0.0)
            continue
        w = np.exp((x - x.max()) / t)
        order = np.argsort(-x, kind="stable")
        if k > 0:
            order = order[:k]
        if p < 1:
            sums = np.cumsum(w[order])
            order = order[:max(1, int(np.searchsorted(sums, p * sums[-1], side="left")) + 1)]
        kept = np.sort(order[(w[order] >= min(least, 1.0)) & (w[order] > 0)])
        sums = np.cumsum(w[kept])
        at = int(np.searchsorted(sums, u * sums[-1], side="right"))
        tokens.append(int(kept[at]))
        logprobs.append(float(np.log(w[kept[at]] / sums[-1])))
    return (torch.tensor(tokens, dtype=torch.int32), torch.tensor(logprobs, dtype=torch.float64))


def exact(case, seed):
    global own
    mine, own = own, False  # the inputs as a checkpoint or a projection gives them, whichever form is timed
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    return {"kv4_attention": _attention_exact, "kv4_append": _append_exact, "norm_rope": _append_exact,
            "sample": _sample_exact}[case["op"]](case, s)
