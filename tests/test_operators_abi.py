"""The decode-step operators' host checks: every refusal, and the calls that have nothing to do, on a
machine without a GPU (fake pointers; no call here reaches a launch)."""
import ctypes

import numpy as np
import pytest

BF16, HAS_ZP, SWIGLU, GEGLU, ADJ, RENORM, K_FULL = 1 << 16, 1 << 3, 1 << 14, 1 << 15, 1 << 17, 1 << 18, 1 << 2
NULL, ALIGN, SHAPE, FLAGS, OVERFLOW, WORKSPACE, GROUP, TYPE, SCHEDULE = 1, 2, 3, 4, 5, 6, 7, 8, 9
P = 0x10000


@pytest.fixture(scope="module")
def w4():
    import weight_only_int4_03_gb300 as w4
    return w4


def staged(st):
    return st >> 16, st & 0xFFFF


def rope_status(w4, **kw):
    a = dict(q=P, ldq=1024, k=P, ldk=1024, v=P, ldv=1024, q_out=P, ldqo=512, kc=P, vc=P, ps=4096, ts=256, hs=128,
             table=P, max_pos=100, pos=P, ld_pos=4, slots=P, status=None, tokens=4, heads=4, kv=2, dim=128,
             rot=128, sections=[64], page=16, n_pages=8, flags=0)
    a.update(kw)
    sec = np.array(a["sections"], np.int32)
    return w4._lib.w4a16_rope_append(
        a["q"], a["ldq"], a["k"], a["ldk"], a["v"], a["ldv"], a["q_out"], a["ldqo"], a["kc"], a["vc"], a["ps"],
        a["ts"], a["hs"], a["table"], a["max_pos"], a["pos"], a["ld_pos"], a["slots"], a["status"], a["tokens"],
        a["heads"], a["kv"], a["dim"], a["rot"], sec.ctypes.data if sec.size else None, sec.size, a["page"],
        a["n_pages"], a["flags"], 0)


@pytest.mark.parametrize("kw,want", [
    (dict(flags=HAS_ZP), (1, FLAGS)),
    (dict(tokens=-1), (1, SHAPE)),
    (dict(heads=-1), (1, SHAPE)),
    (dict(heads=0, kv=0), (1, SHAPE)),
    (dict(dim=0), (1, SHAPE)),
    (dict(rot=0, sections=[0]), (1, SHAPE)),
    (dict(rot=63, sections=[31]), (1, SHAPE)),
    (dict(rot=130, sections=[65]), (1, SHAPE)),
    (dict(max_pos=0), (1, SHAPE)),
    (dict(page=0), (1, SHAPE)),
    (dict(n_pages=0), (1, SHAPE)),
    (dict(sections=[]), (1, SHAPE)),
    (dict(sections=[60, 1, 1, 1, 1]), (1, SHAPE)),
    (dict(sections=[60]), (1, SHAPE)),
    (dict(sections=[80, -16]), (1, SHAPE)),
    (dict(q=None), (1, NULL)), (dict(k=None), (1, NULL)), (dict(v=None), (1, NULL)),
    (dict(q_out=None), (1, NULL)), (dict(kc=None), (1, NULL)), (dict(vc=None), (1, NULL)),
    (dict(table=None), (1, NULL)), (dict(pos=None), (1, NULL)), (dict(slots=None), (1, NULL)),
    (dict(ldq=511), (1, SHAPE)), (dict(ldqo=511), (1, SHAPE)), (dict(ldk=255), (1, SHAPE)),
    (dict(ldv=255), (1, SHAPE)), (dict(ld_pos=3), (1, SHAPE)), (dict(ts=-1), (1, SHAPE)),
    (dict(q=P + 1), (1, ALIGN)), (dict(vc=P + 1), (1, ALIGN)), (dict(table=P + 2), (1, ALIGN)),
    (dict(pos=P + 2), (1, ALIGN)), (dict(slots=P + 4), (1, ALIGN)), (dict(status=P + 2), (1, ALIGN)),
    (dict(heads=1 << 25, ldq=1 << 30), (1, OVERFLOW)),
    (dict(heads=1 << 20, kv=1, dim=2, rot=2, sections=[1], ldq=1 << 21, ldqo=1 << 21), (1, OVERFLOW)),
])
def test_rope_refusals(w4, kw, want):
    assert staged(rope_status(w4, **kw)) == want


def test_rope_nothing_to_do(w4):
    assert rope_status(w4, tokens=0, q=None, k=None, v=None) == 0


def attention_status(w4, **kw):
    a = dict(q=P, ldq=512, k=P, v=P, ps=4096, ts=256, hs=128, out=P, ldo=512, lse=None, table=P, ld_table=8, lens=P,
             ws=P, ws_bytes=1 << 40, batch=3, heads=4, kv=2, dim=128, page=16, n_pages=9, max_pages=8, window=0,
             flags=0)
    a.update(kw)
    return w4._lib.w4a16_paged_attention(
        a["q"], a["ldq"], a["k"], a["v"], a["ps"], a["ts"], a["hs"], a["out"], a["ldo"], a["lse"], a["table"],
        a["ld_table"], a["lens"], a["ws"], a["ws_bytes"], a["batch"], a["heads"], a["kv"], a["dim"], a["page"],
        a["n_pages"], a["max_pages"], a["window"], ctypes.c_float(0.1), a["flags"], 0)


@pytest.mark.parametrize("kw,want", [
    (dict(flags=ADJ), (1, FLAGS)),
    (dict(batch=-1), (1, SHAPE)), (dict(heads=0), (1, SHAPE)), (dict(kv=0), (1, SHAPE)), (dict(kv=3), (1, SHAPE)),
    (dict(dim=0), (1, SHAPE)), (dict(page=0), (1, SHAPE)), (dict(n_pages=0), (1, SHAPE)),
    (dict(max_pages=0), (1, SHAPE)), (dict(window=-1), (1, SHAPE)),
    (dict(dim=80), (2, SHAPE)), (dict(batch=4097), (2, SHAPE)),
    (dict(q=None), (1, NULL)), (dict(k=None), (1, NULL)), (dict(v=None), (1, NULL)), (dict(out=None), (1, NULL)),
    (dict(table=None), (1, NULL)), (dict(lens=None), (1, NULL)), (dict(ws=None), (1, NULL)),
    (dict(ldq=504), (1, SHAPE)), (dict(ldo=504), (1, SHAPE)), (dict(ld_table=7), (1, SHAPE)),
    (dict(hs=-128), (1, SHAPE)),
    (dict(ldq=516), (1, ALIGN)), (dict(ldo=516), (1, ALIGN)), (dict(ts=260), (1, ALIGN)), (dict(q=P + 8), (1, ALIGN)),
    (dict(k=P + 8), (1, ALIGN)), (dict(v=P + 2), (1, ALIGN)), (dict(out=P + 8), (1, ALIGN)),
    (dict(lse=P + 2), (1, ALIGN)), (dict(table=P + 1), (1, ALIGN)), (dict(ws=P + 64), (1, ALIGN)),
    (dict(max_pages=1 << 28, ld_table=1 << 28), (1, OVERFLOW)),
    (dict(batch=4096, max_pages=1 << 26, ld_table=1 << 26), (1, OVERFLOW)),
    (dict(heads=1 << 23, kv=1 << 23, ldq=1 << 30, ldo=1 << 30), (1, OVERFLOW)),
])
def test_attention_refusals(w4, kw, want):
    assert staged(attention_status(w4, **kw)) == want


def test_attention_nothing_to_do_and_workspace(w4):
    assert attention_status(w4, batch=0, q=None, ws=None) == 0
    size = w4.w4a16_paged_attention_workspace_size
    assert size(3, 4, 2, 128, 152) > 0
    assert size(3, 4, 3, 128, 152) == 0 and size(3, 4, 2, 96, 152) == 0 and size(5000, 4, 2, 128, 152) == 0


def moe_status(w4, **kw):
    a = dict(x=P, ldx=512, router=P, up=P, us=P, uz=None, down=P, ds=P, dz=None, res=None, ldr=512, y=P, ldy=512,
             ids=None, tw=None, ws=P, ws_bytes=1 << 40, tokens=3, hidden=512, inter=384, experts=8, top=2, gs=128,
             wt=5, flags=SWIGLU)
    a.update(kw)
    return w4._lib.w4a16_moe_layer(
        a["x"], a["ldx"], a["router"], a["up"], a["us"], a["uz"], a["down"], a["ds"], a["dz"], a["res"], a["ldr"],
        a["y"], a["ldy"], a["ids"], a["tw"], a["ws"], a["ws_bytes"], a["tokens"], a["hidden"], a["inter"],
        a["experts"], a["top"], a["gs"], a["wt"], a["flags"], 0)


@pytest.mark.parametrize("kw,want", [
    (dict(wt=8), (1, TYPE)), (dict(wt=0), (1, TYPE)),
    (dict(flags=0), (1, FLAGS)), (dict(flags=SWIGLU | GEGLU), (1, FLAGS)), (dict(flags=SWIGLU | 1 << 10), (1, FLAGS)),
    (dict(flags=SWIGLU | HAS_ZP), (1, FLAGS)), (dict(wt=4), (1, FLAGS)), (dict(uz=P), (1, FLAGS)),
    (dict(wt=4, flags=SWIGLU | HAS_ZP, uz=P), (1, FLAGS)), (dict(wt=4, flags=SWIGLU | HAS_ZP, dz=P), (1, FLAGS)),
    (dict(tokens=-1), (1, SHAPE)), (dict(hidden=0), (1, SHAPE)), (dict(inter=-128), (1, SHAPE)),
    (dict(experts=0), (1, SCHEDULE)), (dict(top=0), (1, SCHEDULE)), (dict(top=9), (1, SCHEDULE)),
    (dict(tokens=65), (2, SHAPE)), (dict(hidden=384), (2, SHAPE)), (dict(inter=320), (2, SHAPE)),
    (dict(experts=513), (2, SCHEDULE)), (dict(experts=100, top=17), (2, SCHEDULE)),
    (dict(gs=0), (1, GROUP)), (dict(gs=32), (1, GROUP)), (dict(gs=256), (1, GROUP)), (dict(gs=-2), (1, GROUP)),
    (dict(x=None), (1, NULL)), (dict(router=None), (1, NULL)), (dict(up=None), (1, NULL)), (dict(us=None), (1, NULL)),
    (dict(down=None), (1, NULL)), (dict(ds=None), (1, NULL)), (dict(y=None), (1, NULL)), (dict(ws=None), (1, NULL)),
    (dict(ldx=504), (1, SHAPE)), (dict(ldy=504), (1, SHAPE)), (dict(res=P, ldr=504), (1, SHAPE)),
    (dict(ldx=516), (1, ALIGN)), (dict(ldy=516), (1, ALIGN)), (dict(res=P, ldr=516), (1, ALIGN)),
    (dict(x=P + 8), (1, ALIGN)), (dict(router=P + 2), (1, ALIGN)), (dict(up=P + 4), (1, ALIGN)),
    (dict(res=P + 8), (1, ALIGN)), (dict(y=P + 8), (1, ALIGN)), (dict(ids=P + 2), (1, ALIGN)),
    (dict(tw=P + 1), (1, ALIGN)), (dict(ws=P + 16), (1, ALIGN)),
    (dict(ws_bytes=1000), (1, WORKSPACE)),
    (dict(hidden=1 << 21, ldx=1 << 21, ldy=1 << 21), (1, OVERFLOW)),
])
def test_moe_layer_refusals(w4, kw, want):
    assert staged(moe_status(w4, **kw)) == want


def test_moe_layer_nothing_to_do_and_workspace(w4):
    assert moe_status(w4, tokens=0, x=None, ws=None, flags=GEGLU | BF16 | RENORM | K_FULL) == 0
    size = w4.w4a16_moe_layer_workspace_size
    assert size(3, 512, 384, 8, 2) > 0
    assert size(65, 512, 384, 8, 2) == 0 and size(3, 500, 384, 8, 2) == 0 and size(3, 512, 384, 8, 9) == 0
    # Enough for the pairs' activations (two rows each) and outputs.
    assert size(64, 512, 384, 8, 2) >= 128 * (384 * 4 + 512 * 4)


# Heads too wide for one launch: refused after every look at a pointer, before any at the device.
@pytest.mark.parametrize("kw", [
    dict(heads=1 << 20, kv=0, k=P + 1, v=P + 1, kc=P + 1, vc=P + 1, slots=P + 1, page=0, n_pages=-1),
    dict(heads=1 << 20, kv=0, k=None, v=None, kc=None, vc=None, slots=None),
    dict(heads=0, kv=1 << 19, q=P + 1, q_out=P + 1),
], ids=("q_alone_odd", "q_alone_null", "kv_alone_odd"))
def test_rope_pointers_of_absent_heads_are_not_looked_at(w4, kw):
    wide = dict(dim=1024, rot=1024, sections=[512], ldq=1 << 30, ldqo=1 << 30, ldk=1 << 30, ldv=1 << 30)
    assert staged(rope_status(w4, **{**wide, **kw})) == (1, OVERFLOW)


@pytest.mark.parametrize("hidden,inter,experts,top", [(2048, 768, 128, 8), (4096, 14336, 8, 2), (256, 128, 1, 1),
                                                      (512, 256, 60, 5), (256, 128, 512, 16)])
def test_moe_layer_workspace_never_shrinks_with_tokens(w4, hidden, inter, experts, top):
    """A workspace for the most tokens of a program serves its smaller calls."""
    sizes = [w4.w4a16_moe_layer_workspace_size(t, hidden, inter, experts, top) for t in range(1, 65)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
