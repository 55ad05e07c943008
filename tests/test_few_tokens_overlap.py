"""gptq_gemv, gptq_gemv_gated and gptq_moe_layer refuse a result in X's memory (no GPU work: nothing is launched)."""
import ctypes

import pytest

import post_weight_quantization_21_amd as gq

P = 0x100000  # a made-up aligned address
SQUARE = gq.Packed(P, P, P, None, 128, 128, 4, 32)
R = ctypes.byref(SQUARE)


def calls(Y, yd=gq.DT_BF16, M=3, ldx=256, ldy=256):
    lib = gq.load_library()
    ws = gq.moe_workspace_bytes(M, 128, 128, 4, 2)
    yield lib.gptq_gemv(P, gq.DT_BF16, M, ldx, R, None, Y, yd, ldy, None, 0, None)
    yield lib.gptq_gemv_gated(P, gq.DT_BF16, M, ldx, R, R, Y, yd, ldy, None, 0, None)
    yield lib.gptq_moe_layer(P, gq.DT_BF16, M, ldx, P, gq.DT_F32, 4, 2, 1, R, R, R, P, P, Y, yd, ldy, P, ws, None)


@pytest.mark.parametrize("kw", [
    dict(Y=P),                                        # in place
    dict(Y=P, M=1),
    dict(Y=P + 2 * 255),                              # one element at X's next row
    dict(Y=P + 2 * 512, ldy=128),                     # from X's last row on
    dict(Y=P - 2 * 256 * 2 - 2 * 127, M=3),           # its last row ends in X's first
    dict(Y=P + 2 * 128, yd=gq.DT_F32, ldy=128),       # wider values between X's rows: 512 bytes for 256
    dict(Y=P + 2 * 128, ldy=264),                     # between the rows, but at another pitch
])
def test_refused(kw):
    for status in calls(**kw):
        assert status == gq.ERR_INVALID_ARG and b"overlap" in gq.load_library().gptq_last_error()
