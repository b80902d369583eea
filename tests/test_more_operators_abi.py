"""Host checks of the norms with rotation, the cache held in 4 bits and sampling: every refusal, and the calls that
have nothing to do, on a machine without a GPU (fake pointers; no call here reaches a launch), through ctypes and
through the extension module."""
import os

import numpy as np
import pytest

BF16, HAS_ZP, ADJ = 1 << 16, 1 << 3, 1 << 17
NULL, ALIGN, SHAPE, FLAGS, OVERFLOW, WORKSPACE, GROUP = 1, 2, 3, 4, 5, 6, 7
P = 0x10000


@pytest.fixture(scope="module")
def w4():
    import weight_only_int4_03_gb300 as w4
    return w4


def staged(st):
    return st >> 16, st & 0xFFFF


def status(w4, name, args):
    """The entry's status, the same through each way of calling it."""
    direct = {"w4a16_norm_rope_append": w4._norm_rope_append, "w4a16_kv4_append": w4._kv4_append,
              "w4a16_kv4_attention": w4._kv4_attention, "w4a16_sample": w4._sample}[name]
    ways = [w4._through_ctypes(name)] + ([direct] if os.path.exists(w4.CALL_PATH) else [])
    got = {way(*args) for way in ways}
    assert len(got) == 1
    return staged(got.pop())


COMMON = dict(q=P, ldq=1024, k=P, ldk=1024, v=P, ldv=1024, qn=P, kn=P, eps=1e-6, q_out=P, ldqo=512, table=P, max_pos=100,
              pos=P, ld_pos=4, slots=P, status=None, tokens=4, heads=4, kv=2, dim=128, rot=128, sections=[64], page=16,
              n_pages=8, flags=0)


def norm_status(w4, **kw):
    a = dict(COMMON, kc=P, vc=P, ps=4096, ts=256, hs=128)
    a.update(kw)
    sec = np.array(a["sections"], np.int32)
    return status(w4, "w4a16_norm_rope_append", [
        a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["qn"], a["kn"], a["eps"], a["q_out"], a["ldqo"], a["kc"],
        a["vc"], a["ps"], a["ts"], a["hs"], a["table"], a["max_pos"], a["pos"], a["ld_pos"], a["slots"], a["status"],
        a["tokens"], a["heads"], a["kv"], a["dim"], a["rot"], sec.ctypes.data if sec.size else None, sec.size, a["page"],
        a["n_pages"], a["flags"], 0])


def append_status(w4, **kw):
    a = dict(COMMON, cache=P, stride=2 * 16 * 136, ko=P, ldko=256, vo=P, ldvo=256, gs=-1)
    a.update(kw)
    sec = np.array(a["sections"], np.int32)
    return status(w4, "w4a16_kv4_append", [
        a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["qn"], a["kn"], a["eps"], a["q_out"], a["ldqo"], a["cache"],
        a["stride"], a["ko"], a["ldko"], a["vo"], a["ldvo"], a["table"], a["max_pos"], a["pos"], a["ld_pos"], a["slots"],
        a["status"], a["tokens"], a["heads"], a["kv"], a["dim"], a["rot"], sec.ctypes.data if sec.size else None, sec.size,
        a["page"], a["n_pages"], a["gs"], a["flags"], 0])


BOTH = [
    (dict(flags=HAS_ZP), (1, FLAGS)), (dict(tokens=-1), (1, SHAPE)), (dict(heads=-1), (1, SHAPE)), (dict(kv=-1), (1, SHAPE)),
    (dict(dim=0), (1, SHAPE)), (dict(rot=-2, sections=[]), (1, SHAPE)), (dict(rot=63, sections=[31]), (1, SHAPE)),
    (dict(rot=130, sections=[65]), (1, SHAPE)), (dict(rot=0), (1, SHAPE)), (dict(sections=[]), (1, SHAPE)),
    (dict(sections=[60, 1, 1, 1, 1]), (1, SHAPE)), (dict(sections=[60]), (1, SHAPE)), (dict(sections=[80, -16]), (1, SHAPE)),
    (dict(max_pos=0), (1, SHAPE)), (dict(page=0), (1, SHAPE)), (dict(n_pages=0), (1, SHAPE)),
    (dict(eps=-1e-6), (1, SHAPE)), (dict(eps=float("nan")), (1, SHAPE)), (dict(eps=float("inf")), (1, SHAPE)),
    (dict(q=None), (1, NULL)), (dict(k=None), (1, NULL)), (dict(v=None), (1, NULL)), (dict(q_out=None), (1, NULL)),
    (dict(table=None), (1, NULL)), (dict(pos=None), (1, NULL)), (dict(slots=None), (1, NULL)),
    (dict(ldq=511), (1, SHAPE)), (dict(ldqo=511), (1, SHAPE)), (dict(ldk=255), (1, SHAPE)), (dict(ldv=255), (1, SHAPE)),
    (dict(ld_pos=3), (1, SHAPE)),
    (dict(q=P + 1), (1, ALIGN)), (dict(qn=P + 1), (1, ALIGN)), (dict(kn=P + 1), (1, ALIGN)), (dict(table=P + 2), (1, ALIGN)),
    (dict(pos=P + 2), (1, ALIGN)), (dict(slots=P + 4), (1, ALIGN)), (dict(status=P + 2), (1, ALIGN)),
]


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(heads=0, kv=0), (1, SHAPE)), (dict(kc=None), (1, NULL)), (dict(vc=None), (1, NULL)), (dict(ts=-1), (1, SHAPE)),
    (dict(kc=P + 1), (1, ALIGN)), (dict(heads=1 << 25, ldq=1 << 30), (1, OVERFLOW)),
])
def test_norm_rope_refusals(w4, kw, want):
    assert norm_status(w4, **kw) == want


@pytest.mark.parametrize("kw,want", BOTH + [
    (dict(kv=0), (1, SHAPE)), (dict(dim=96, rot=96, sections=[48]), (2, SHAPE)), (dict(dim=512, rot=128), (2, SHAPE)),
    (dict(rot=24, sections=[12]), (2, SHAPE)), (dict(page=65537), (2, SHAPE)), (dict(gs=32), (1, GROUP)), (dict(gs=0), (1, GROUP)),
    (dict(gs=-2), (1, GROUP)), (dict(gs=256), (1, GROUP)), (dict(gs=192), (1, GROUP)), (dict(cache=None), (1, NULL)),
    (dict(stride=2 * 16 * 136 - 16), (1, SHAPE)), (dict(stride=-16), (1, SHAPE)), (dict(gs=64), (1, SHAPE)),
    (dict(ldko=255), (1, SHAPE)), (dict(ldvo=255), (1, SHAPE)),
    (dict(stride=2 * 16 * 136 + 8), (1, ALIGN)), (dict(cache=P + 8), (1, ALIGN)), (dict(ko=P + 8), (1, ALIGN)),
    (dict(vo=P + 2), (1, ALIGN)), (dict(ldko=260), (1, ALIGN)), (dict(ldvo=260), (1, ALIGN)), (dict(ldq=1028), (1, ALIGN)),
    (dict(ldk=1028), (1, ALIGN)), (dict(ldv=1028), (1, ALIGN)), (dict(ldqo=516), (1, ALIGN)), (dict(q=P + 8), (1, ALIGN)),
    (dict(k=P + 8), (1, ALIGN)), (dict(v=P + 8), (1, ALIGN)), (dict(q_out=P + 8), (1, ALIGN)), (dict(qn=P + 8), (1, ALIGN)),
    (dict(kn=P + 8), (1, ALIGN)), (dict(table=P + 8), (1, ALIGN)),
])
def test_kv4_append_refusals(w4, kw, want):
    assert append_status(w4, **kw) == want


def test_nothing_to_append(w4):
    none = dict(tokens=0, q=None, k=None, v=None, slots=None)
    assert norm_status(w4, **none) == (0, 0)
    assert append_status(w4, **none, cache=None) == (0, 0)
    # What absent heads or an absent rotation would use is not looked at: these are refused for their width alone.
    wide = dict(heads=(1 << 20) + 1, dim=1024, rot=0, sections=[], ldq=1 << 30, ldqo=1 << 30)
    assert norm_status(w4, **wide, kv=0, k=P + 1, v=None, kc=P + 1, vc=None, slots=P + 1, kn=P + 1, table=P + 1, pos=None,
                       max_pos=0, page=0) == (1, OVERFLOW)


def attention_status(w4, **kw):
    a = dict(q=P, ldq=512, cache=P, stride=2 * 16 * 136, out=P, ldo=512, lse=None, table=P, ld_table=8, lens=P, ws=P,
             ws_bytes=1 << 40, batch=3, heads=4, kv=2, dim=128, page=16, n_pages=9, max_pages=8, gs=-1, window=0, flags=0)
    a.update(kw)
    return status(w4, "w4a16_kv4_attention", [
        a["q"], a["ldq"], a["cache"], a["stride"], a["out"], a["ldo"], a["lse"], a["table"], a["ld_table"], a["lens"], a["ws"],
        a["ws_bytes"], a["batch"], a["heads"], a["kv"], a["dim"], a["page"], a["n_pages"], a["max_pages"], a["gs"],
        a["window"], 0.1, a["flags"], 0])


@pytest.mark.parametrize("kw,want", [
    (dict(flags=ADJ), (1, FLAGS)),
    (dict(batch=-1), (1, SHAPE)), (dict(heads=0), (1, SHAPE)), (dict(kv=0), (1, SHAPE)), (dict(kv=3), (1, SHAPE)),
    (dict(dim=0), (1, SHAPE)), (dict(page=0), (1, SHAPE)), (dict(n_pages=0), (1, SHAPE)), (dict(max_pages=0), (1, SHAPE)),
    (dict(window=-1), (1, SHAPE)), (dict(dim=96), (2, SHAPE)), (dict(batch=4097), (2, SHAPE)), (dict(page=65537), (2, SHAPE)),
    (dict(gs=32), (1, GROUP)), (dict(gs=256), (1, GROUP)), (dict(gs=0), (1, GROUP)),
    (dict(q=None), (1, NULL)), (dict(cache=None), (1, NULL)), (dict(out=None), (1, NULL)), (dict(table=None), (1, NULL)),
    (dict(lens=None), (1, NULL)), (dict(ws=None), (1, NULL)),
    (dict(ldq=504), (1, SHAPE)), (dict(ldo=504), (1, SHAPE)), (dict(ld_table=7), (1, SHAPE)),
    (dict(stride=2 * 16 * 136 - 16), (1, SHAPE)), (dict(gs=64), (1, SHAPE)),
    (dict(ldq=516), (1, ALIGN)), (dict(ldo=516), (1, ALIGN)), (dict(stride=2 * 16 * 136 + 8), (1, ALIGN)),
    (dict(q=P + 8), (1, ALIGN)), (dict(cache=P + 8), (1, ALIGN)), (dict(out=P + 8), (1, ALIGN)), (dict(lse=P + 2), (1, ALIGN)),
    (dict(table=P + 1), (1, ALIGN)), (dict(lens=P + 2), (1, ALIGN)), (dict(ws=P + 64), (1, ALIGN)),
    (dict(max_pages=1 << 28, ld_table=1 << 28), (1, OVERFLOW)),
    (dict(batch=4096, max_pages=1 << 26, ld_table=1 << 26), (1, OVERFLOW)),
    (dict(heads=1 << 23, kv=1 << 23, ldq=1 << 30, ldo=1 << 30), (1, OVERFLOW)),
])
def test_kv4_attention_refusals(w4, kw, want):
    assert attention_status(w4, **kw) == want


def test_sizes_of_cache_and_workspace(w4):
    assert attention_status(w4, batch=0, q=None, ws=None) == (0, 0)
    size = w4.w4a16_kv4_attention_workspace_size
    assert size(3, 4, 2, 128, 152) > 0
    assert size(3, 4, 3, 128, 152) == 0 and size(3, 4, 2, 96, 152) == 0 and size(5000, 4, 2, 128, 152) == 0
    record = w4.w4a16_kv4_record_bytes
    assert record(16, 128, -1) == record(16, 128, 128) == 16 * 136 and record(16, 128, 64) == 16 * 144
    assert record(1, 64, -1) == 80 and record(3, 64, 64) == 224 and record(65536, 256, 64) == 65536 * 288
    assert record(0, 128, -1) == record(65537, 128, -1) == record(16, 96, -1) == record(16, 128, 32) == 0
    assert record(16, 128, 256) == record(-1, 64, -1) == 0


def sample_status(w4, **kw):
    a = dict(logits=P, ld=1000, u=P, t=P, k=P, p=P, m=P, tokens=P, logs=P, status=P, batch=2, vocab=1000, flags=0)
    a.update(kw)
    return status(w4, "w4a16_sample", [a[n] for n in ("logits", "ld", "u", "t", "k", "p", "m", "tokens", "logs", "status",
                                                     "batch", "vocab", "flags")] + [0])


@pytest.mark.parametrize("kw,want", [
    (dict(flags=HAS_ZP), (1, FLAGS)), (dict(batch=-1), (1, SHAPE)), (dict(vocab=0), (1, SHAPE)), (dict(ld=999), (1, SHAPE)),
    (dict(vocab=524289, ld=1 << 20), (2, SHAPE)), (dict(batch=(1 << 24) + 1), (2, SHAPE)),
    (dict(logits=None), (1, NULL)), (dict(u=None), (1, NULL)), (dict(tokens=None), (1, NULL)),
    (dict(logits=P + 1), (1, ALIGN)), (dict(u=P + 2), (1, ALIGN)), (dict(t=P + 2), (1, ALIGN)), (dict(k=P + 2), (1, ALIGN)),
    (dict(p=P + 1), (1, ALIGN)), (dict(m=P + 2), (1, ALIGN)), (dict(tokens=P + 2), (1, ALIGN)), (dict(logs=P + 2), (1, ALIGN)),
    (dict(status=P + 2), (1, ALIGN)),
])
def test_sample_refusals(w4, kw, want):
    assert sample_status(w4, **kw) == want


def test_nothing_to_sample(w4):
    assert sample_status(w4, batch=0, logits=None, u=None, tokens=None) == (0, 0)


def test_wrappers_raise_the_library_error(w4):
    for call, want in (
        (lambda: w4.w4a16_norm_rope_append(P, P, P, P, P, 0.0, P, P, P, P, P, P, None, 4, 4, 2, 128, 128, [60], 100, 16, 8,
                                           stream=0), (1, SHAPE)),
        (lambda: w4.w4a16_kv4_append(P, P, P, P, P, 0.0, P, P, P, P, P, None, 4, 4, 2, 128, 128, [64], 100, 16, 8, 32,
                                     stream=0), (1, GROUP)),
        (lambda: w4.w4a16_kv4_attention(P, P, P, P, P, None, 3, 4, 2, 128, 16, 9, 8, -1, 0.1, stream=0), (1, NULL)),
        (lambda: w4.w4a16_sample(P, P, P, 2, 1000, flags=1 << 30, stream=0), (1, FLAGS)),
    ):
        with pytest.raises(w4.W4A16Error) as e:
            call()
        assert staged(e.value.status) == want
