"""The paged cache held in 4 bits as its documentation describes it, in plain torch: reading it, and coding values."""
import torch

TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
UNIT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}


def groups_of(dim, group_size):
    return 1 if group_size == -1 else dim // group_size


def word_places(dim):
    """Places of the words of a row: (keys, values)."""
    blocks, keys, values = dim // 64, [], []
    for w in range(dim // 8):
        b, t, i, g = w // 8, w % 8 // 2, w % 2, w % 8
        keys.append(w if blocks == 1 else 16 * (b // 2) + 4 * t + 2 * (b % 2) + i)
        values.append(g * blocks + b)
    return keys, values


def read(cache, page, kv, dim, group_size, dtype):
    """cache [n_pages, bytes] uint8 -> codes [2, n_pages, page, kv, dim] and (s, b) [2, n_pages, page, kv, groups, 2]."""
    groups = groups_of(dim, group_size)
    record = (page * (dim + 8 * groups) + 15) // 16 * 16
    rec = cache[:, :kv * record].reshape(-1, kv, record)
    codes, params = [], []
    for side, places in enumerate(word_places(dim)):
        at = side * page * dim // 2
        words = rec[:, :, at:at + page * dim // 2].contiguous().view(torch.int32).view(-1, kv, page, dim // 8)
        words = words[..., torch.tensor(places, device=cache.device)]
        shift = torch.arange(0, 32, 4, device=cache.device, dtype=torch.int32)
        codes.append(((words.unsqueeze(-1) >> shift) & 15).flatten(-2).transpose(1, 2))
        at = page * dim + side * page * groups * 4
        sb = rec[:, :, at:at + page * groups * 4].contiguous().view(TYPES[dtype]).view(-1, kv, page, groups, 2)
        params.append(sb.transpose(1, 2))
    return torch.stack(codes), torch.stack(params)


def values(codes, params):
    """What the codes stand for, in 64 bits."""
    x = codes.unflatten(-1, (params.shape[-2], -1)).double()
    return (x * params[..., 0].double().unsqueeze(-1) + params[..., 1].double().unsqueeze(-1)).flatten(-2)


def coded(x, group_size, dtype):
    """x [..., dim] of the cache's type, coded by the definition in fp32 (every step of it is one IEEE operation)."""
    x = x.float().unflatten(-1, (groups_of(x.shape[-1], group_size), -1))
    lo, hi = x.amin(-1), x.amax(-1)
    s, b = ((hi - lo) / 15).to(TYPES[dtype]), lo.to(TYPES[dtype])
    sf, bf = s.float().unsqueeze(-1), b.float().unsqueeze(-1)
    q = torch.where(sf > 0, ((x - bf) / sf).round().clamp(0, 15), torch.zeros_like(x))
    return q.int().flatten(-2), torch.stack((s, b), -1)
