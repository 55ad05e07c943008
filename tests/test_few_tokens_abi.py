"""gptq_gemv, gptq_gemv_gated and gptq_moe_layer: workspace queries and refused calls (no GPU work: every refusal
comes before anything is launched, and so do the calls without tokens)."""
import ctypes

import pytest

import post_weight_quantization_21_amd as gq

P = 0x10000  # a made-up aligned address


def packed(d_out=64, d_in=128, bits=4, group=32, at=P, scales=P, zeros=P, kperm=None):
    return gq.Packed(at, scales, zeros, kperm, d_out, d_in, bits, group)


def gemv(w, X=P, xd=gq.DT_BF16, M=1, ldx=128, bias=None, Y=P, yd=gq.DT_BF16, ldy=64, ws=P, ws_bytes=1 << 20):
    return gq.load_library().gptq_gemv(X, xd, M, ldx, None if w is None else ctypes.byref(w), bias, Y, yd, ldy, ws, ws_bytes, None)


def gated(a, b, M=1, ldx=128, ldh=64, ws=P, ws_bytes=1 << 20):
    return gq.load_library().gptq_gemv_gated(P, gq.DT_F16, M, ldx, ctypes.byref(a), ctypes.byref(b), P, gq.DT_F16, ldh, ws, ws_bytes, None)


def moe(gate, up, down, T=2, X=P, xd=gq.DT_BF16, ldx=128, router=P, rd=gq.DT_F32, E=4, k=2, ids=P, weights=P, Y=P,
        yd=gq.DT_F32, ldy=128, ws=P, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = 1 << 30
    r = [None if w is None else ctypes.byref(w) for w in (gate, up, down)]
    return gq.load_library().gptq_moe_layer(X, xd, T, ldx, router, rd, E, k, 1, *r, ids, weights, Y, yd, ldy, ws, ws_bytes, None)


def message():
    return gq.load_library().gptq_last_error()


@pytest.mark.parametrize("w,status,text", [
    (None, gq.ERR_INVALID_ARG, b"NULL"),
    (packed(d_out=0), gq.ERR_INVALID_ARG, b"sizes"),
    (packed(d_in=0), gq.ERR_INVALID_ARG, b"sizes"),
    (packed(bits=1), gq.ERR_INVALID_ARG, b"bits"),
    (packed(bits=9), gq.ERR_INVALID_ARG, b"bits"),
    (packed(bits=5), gq.ERR_UNSUPPORTED, b"bits"),
    (packed(group=48), gq.ERR_INVALID_ARG, b"group_size"),
    (packed(group=-32), gq.ERR_INVALID_ARG, b"group_size"),
    (packed(group=16), gq.ERR_UNSUPPORTED, b"multiples of 32"),
    (packed(d_in=48, group=0), gq.ERR_UNSUPPORTED, b"multiples of 32"),
    (packed(d_in=(1 << 20) + 32, group=32), gq.ERR_UNSUPPORTED, b"2^20"),
    (packed(d_out=(1 << 28) + 1), gq.ERR_UNSUPPORTED, b"2^28"),
    (packed(at=None), gq.ERR_INVALID_ARG, b"NULL"),
    (packed(scales=None), gq.ERR_INVALID_ARG, b"NULL"),
    (packed(zeros=None), gq.ERR_INVALID_ARG, b"NULL"),
    (packed(at=P + 8), gq.ERR_INVALID_ARG, b"aligned"),
    (packed(scales=P + 2), gq.ERR_INVALID_ARG, b"aligned"),
    (packed(kperm=P + 1), gq.ERR_INVALID_ARG, b"aligned"),
])
def test_packed_layers_refused(w, status, text):
    assert gemv(w, ldx=1 << 21, ldy=1 << 31) == status
    assert text in message()
    good = packed()
    if w is not None:
        assert gated(good, w) != gq.OK and gated(w, good) != gq.OK
        assert moe(good, good, w) != gq.OK


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), gq.ERR_INVALID_ARG), (dict(M=17), gq.ERR_UNSUPPORTED),
    (dict(xd=gq.DT_F32), gq.ERR_INVALID_ARG), (dict(yd=7), gq.ERR_INVALID_ARG), (dict(xd=9), gq.ERR_INVALID_ARG),
    (dict(X=None), gq.ERR_INVALID_ARG), (dict(Y=None), gq.ERR_INVALID_ARG),
    (dict(ldx=120), gq.ERR_INVALID_ARG), (dict(ldx=132), gq.ERR_INVALID_ARG), (dict(ldy=63), gq.ERR_INVALID_ARG),
    (dict(X=P + 8), gq.ERR_INVALID_ARG), (dict(Y=P + 1), gq.ERR_INVALID_ARG), (dict(Y=P + 2, yd=gq.DT_F32), gq.ERR_INVALID_ARG),
    (dict(bias=P + 2), gq.ERR_INVALID_ARG),
])
def test_gemv_arguments_refused(kw, status):
    assert gemv(packed(), **kw) == status


def test_gemv_workspace():
    need = gq.workspace_bytes(gq.OP_GEMV, 64, 4128, 3)
    assert need >= 3 * 4608 * 2  # whole quads of columns
    ordered = packed(d_in=4128, group=0, kperm=P)
    assert gemv(ordered, M=3, ldx=4128, ws_bytes=need - 1) == gq.ERR_WORKSPACE
    assert gemv(ordered, M=3, ldx=4128, ws=None) == gq.ERR_WORKSPACE
    assert gemv(ordered, M=3, ldx=4128, ws=P + 8) == gq.ERR_INVALID_ARG
    assert gated(ordered, ordered, M=3, ldx=4128, ws_bytes=need - 1) == gq.ERR_WORKSPACE
    for m, d in ((1, gq.GEMV_GATHERS), (16, gq.GEMV_GATHERS // 16)):  # the largest without one, and one unit more
        assert gq.workspace_bytes(gq.OP_GEMV, 64, d, m) == 0 < gq.workspace_bytes(gq.OP_GEMV, 64, d + 32, m)
    with pytest.raises(gq.GptqError) as ei:
        gq.workspace_bytes(9, 1, 1)  # the number between the operations stays free
    assert ei.value.status == gq.ERR_INVALID_ARG


def test_no_tokens_is_no_work():
    assert gemv(packed(), X=None, Y=None, M=0) == gq.OK
    assert gated(packed(), packed(), M=0) == gq.OK
    down = packed(d_out=128, d_in=64)
    assert moe(packed(), packed(), down, T=0, X=None, Y=None, ids=None, weights=None, ws=None) == gq.OK


@pytest.mark.parametrize("other", [packed(d_out=65), packed(d_in=160), packed(bits=8), packed(group=64), packed(kperm=P)])
def test_gate_and_up_must_agree(other):
    assert gated(packed(), other, ldx=256, ldh=128) == gq.ERR_INVALID_ARG
    assert b"agree" in message()
    assert moe(packed(), other, packed(d_out=128, d_in=64)) == gq.ERR_INVALID_ARG


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), gq.ERR_INVALID_ARG), (dict(T=17), gq.ERR_UNSUPPORTED), (dict(E=0), gq.ERR_INVALID_ARG),
    (dict(E=513), gq.ERR_UNSUPPORTED), (dict(k=0), gq.ERR_INVALID_ARG), (dict(k=5), gq.ERR_INVALID_ARG),
    (dict(E=40, k=17), gq.ERR_UNSUPPORTED), (dict(xd=gq.DT_F32), gq.ERR_INVALID_ARG), (dict(yd=4), gq.ERR_INVALID_ARG),
    (dict(rd=gq.DT_F16), gq.ERR_INVALID_ARG), (dict(X=None), gq.ERR_INVALID_ARG), (dict(Y=None), gq.ERR_INVALID_ARG),
    (dict(ldx=64), gq.ERR_INVALID_ARG), (dict(ldy=127), gq.ERR_INVALID_ARG), (dict(X=P + 4), gq.ERR_INVALID_ARG),
    (dict(router=None, ids=None), gq.ERR_INVALID_ARG), (dict(router=None, weights=None), gq.ERR_INVALID_ARG),
    (dict(router=P + 8), gq.ERR_INVALID_ARG), (dict(ids=P + 2), gq.ERR_INVALID_ARG), (dict(weights=P + 1), gq.ERR_INVALID_ARG),
    (dict(ws=None), gq.ERR_WORKSPACE), (dict(ws_bytes=1000), gq.ERR_WORKSPACE), (dict(ws=P + 8), gq.ERR_INVALID_ARG),
])
def test_moe_arguments_refused(kw, status):
    assert moe(packed(), packed(), packed(d_out=128, d_in=64), **kw) == status


@pytest.mark.parametrize("down", [packed(), packed(d_out=128, d_in=32), packed(d_out=96, d_in=64), packed(d_out=128, d_in=64, bits=8)])
def test_moe_down_must_fit(down):
    assert moe(packed(), packed(), down) == gq.ERR_INVALID_ARG


def test_moe_workspace_sizes():
    small, large = gq.moe_workspace_bytes(1, 128, 64, 4, 2), gq.moe_workspace_bytes(16, 4096, 14336, 8, 2)
    assert 0 < small < large
    assert large >= 32 * (3 * 14336 * 2 + 4096 * 4)  # h in three pieces and the down product's rows, per pair
    for bad, status in (((17, 128, 64, 4, 2), gq.ERR_UNSUPPORTED), ((1, 0, 64, 4, 2), gq.ERR_INVALID_ARG),
                        ((1, 128, 64, 4, 5), gq.ERR_INVALID_ARG), ((1, 128, 1 << 21, 4, 2), gq.ERR_UNSUPPORTED)):
        with pytest.raises(gq.GptqError) as ei:
            gq.moe_workspace_bytes(*bad)
        assert ei.value.status == status
    assert gq.load_library().gptq_moe_workspace_bytes(1, 128, 64, 4, 2, None) == gq.ERR_INVALID_ARG
