"""The calls with 8-bit floating-point operands refuse bad arguments with a
status before any launch, and their binding refuses tensors that do not fit.
CPU only: no address here is dereferenced."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
A = P(0x10000)
ODD = P(0x10001)
H8 = P(0x10008)
NULL, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 6
BIG = 1 << 20


@pytest.fixture(scope="module")
def L():
    from mmvq_q2_gb300 import build
    build.build()
    import mmvq_q2_gb300 as q
    return q.lib()


def refused(fn, good, cases):
    for change, status in cases:
        args = list(good)
        for i, v in change.items():
            args[i] = v
        assert fn(*args) == status, change


def test_quantize_refusals(L):
    # x, type, rows, K, ldx, block_rows, q, ldq, scales, ld_scales, stream
    good = (A, 0, 5, 300, 300, 1, A, 300, A, 3, None)
    refused(L.fp8_quantize, good, [
        ({0: None}, NULL), ({6: None}, NULL), ({8: None}, NULL),
        ({1: 2}, SHAPE), ({2: -1}, SHAPE), ({2: (1 << 30) + 1}, SHAPE), ({3: 0}, SHAPE),
        ({3: BIG + 1, 4: BIG + 1, 7: BIG + 1, 9: BIG}, SHAPE), ({4: 299}, SHAPE), ({5: 0}, SHAPE), ({5: 64}, SHAPE),
        ({7: 299}, SHAPE), ({9: 2}, SHAPE), ({0: ODD}, ALIGN), ({0: P(0x10002)}, ALIGN), ({8: P(0x10002)}, ALIGN),
    ])


def test_swiglu_refusals(L):
    # gate_up, type, rows, N, ld, q, ldq, scales, ld_scales, stream
    good = (A, 1, 5, 300, 600, A, 300, A, 3, None)
    refused(L.swiglu_fp8_rows, good, [
        ({0: None}, NULL), ({5: None}, NULL), ({7: None}, NULL),
        ({1: -1}, SHAPE), ({2: -1}, SHAPE), ({3: 0}, SHAPE), ({4: 599}, SHAPE), ({6: 299}, SHAPE), ({8: 2}, SHAPE),
        ({3: BIG // 2 + 1, 4: 2 * BIG, 6: BIG, 8: BIG}, SHAPE), ({0: ODD}, ALIGN), ({7: ODD}, ALIGN),
    ])


def test_gemm_refusals(L):
    # x, m, K, ldx, x_scales, ld_xs, W, N, w_scales, y, y_type, ldy, stream
    good = (A, 3, 272, 272, A, 3, A, 100, A, A, 0, 100, None)
    refused(L.fp8_gemm, good, [
        ({0: None}, NULL), ({4: None}, NULL), ({6: None}, NULL), ({8: None}, NULL), ({9: None}, NULL),
        ({1: -1}, SHAPE), ({1: 1 << 30}, SHAPE), ({2: 0}, SHAPE), ({2: 264}, SHAPE), ({2: BIG + 16, 3: BIG + 16, 5: BIG}, SHAPE),
        ({3: 256}, SHAPE), ({3: 280}, SHAPE), ({5: 2}, SHAPE), ({7: 0}, SHAPE), ({7: 1 << 30, 11: 1 << 30}, SHAPE),
        ({10: 2}, SHAPE), ({11: 99}, SHAPE),
        ({0: H8}, ALIGN), ({6: H8}, ALIGN), ({4: ODD}, ALIGN), ({8: ODD}, ALIGN), ({9: P(0x10002)}, ALIGN),
        ({9: ODD, 10: 1}, ALIGN),
    ])


def test_moe_refusals(L):
    need = L.fp8_moe_workspace_bytes(3, 2, 272, 144)
    assert need > 0
    for bad in ((-1, 2, 272, 144), (129, 2, 272, 144), (3, 0, 272, 144), (3, 33, 272, 144), (128, 9, 272, 144),
                (3, 2, 264, 144), (3, 2, 0, 144), (3, 2, 16400, 144), (3, 2, 272, 136), (3, 2, 272, 0),
                (3, 2, 272, 16400)):
        assert L.fp8_moe_workspace_bytes(*bad) == 0, bad
    # x, m, dim, ldx, ids, route_w, topk, E, gate_up, gs, down, ds, inter, y, y_type, ldy, workspace, bytes, stream
    good = (A, 3, 272, 272, A, A, 2, 8, A, A, A, A, 144, A, 0, 272, A, need, None)
    refused(L.fp8_moe, good, [
        *[({i: None}, NULL) for i in (0, 4, 5, 8, 9, 10, 11, 13)],
        ({1: -1}, SHAPE), ({1: 129}, SHAPE), ({2: 264}, SHAPE), ({3: 271}, SHAPE), ({6: 0}, SHAPE), ({6: 33}, SHAPE),
        ({7: 0}, SHAPE), ({7: 1025}, SHAPE), ({12: 136}, SHAPE), ({14: 2}, SHAPE), ({15: 271}, SHAPE),
        ({16: None}, WORKSPACE), ({17: need - 1}, WORKSPACE),
        ({0: ODD}, ALIGN), ({4: ODD}, ALIGN), ({5: ODD}, ALIGN), ({8: H8}, ALIGN), ({9: ODD}, ALIGN), ({10: H8}, ALIGN),
        ({11: ODD}, ALIGN), ({13: P(0x10002)}, ALIGN), ({16: P(0x10080)}, ALIGN),
    ])


# ---- the binding -----------------------------------------------------------------

class Fake:
    """What the binding reads off a tensor: no memory, any device."""

    def __init__(self, dtype, *shape, device=0, stride=None):
        self.dtype, self.shape, self.device_index, self.strides = getattr(torch, dtype), shape, device, stride

    def stride(self):
        out, n = [], 1
        for s in reversed(self.shape):
            out.insert(0, n)
            n *= s
        return self.strides or tuple(out)

    def data_ptr(self):
        return 0x10000

    def get_device(self):
        return self.device_index


@pytest.fixture
def calls(L):
    """The binding's native half over functions that do nothing; the current device is 0."""
    import mmvq_q2_gb300 as q
    m = q._calls()
    nothing = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: 0)
    at = ctypes.cast(nothing, P).value
    try:
        m.setup((torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8), (at,) * 6, lambda: 0)
        m.setup_fp8(torch.float8_e4m3fn, (at,) * 5)
        yield m
    finally:
        q._native = None
        q._calls()


F, B, I, U, Q = "float32", "bfloat16", "int32", "uint8", "float8_e4m3fn"
GOOD = {
    "fp8_quantize": [(B, 5, 300), 1, (Q, 5, 300), (F, 5, 3), 0],
    "swiglu_fp8_rows": [(F, 5, 600), 1, (Q, 5, 300), (F, 5, 3), 0],
    "fp8_gemm": [(Q, 5, 272), (F, 5, 3), (Q, 130, 272), (F, 2, 3), (B, 5, 130), 0],
    "fp8_moe": [(B, 5, 272), (I, 5, 2), (F, 5, 2), (Q, 8, 2, 144, 272), (F, 8, 2, 2, 3), (Q, 8, 272, 144),
                (F, 8, 3, 2), (F, 5, 272), (U, 4096), 0],
}
WRONG = {
    "fp8_quantize": [(0, (I, 5, 300)), (0, (B, 1500,)), (2, (U, 5, 300)), (2, (Q, 5, 304)), (3, (F, 5, 2)),
                     (3, (F, 1, 3)), (3, (B, 5, 3)), (0, None)],
    "swiglu_fp8_rows": [(0, (F, 5, 601)), (0, (F, 5, 598)), (2, (Q, 5, 600)), (3, (F, 6, 3))],
    "fp8_gemm": [(0, (U, 5, 272)), (0, (Q, 5, 256)), (1, (F, 5, 2)), (1, (F, 3, 5)), (2, (Q, 130, 256)), (3, (F, 1, 3)),
                 (3, (F, 2, 2)), (3, (F, 6)), (4, (B, 5, 131)), (4, (I, 5, 130)), (4, None)],
    "fp8_moe": [(0, (F, 5, 272)), (1, (I, 5, 3)), (1, ("int64", 5, 2)), (1, (I, 10)), (2, (F, 4, 2)), (2, (B, 5, 2)),
                (3, (Q, 8, 288, 272)), (3, (Q, 7, 2, 144, 272)), (3, (Q, 8, 2, 128, 272)), (4, (F, 8, 2, 2, 2)),
                (4, (F, 8, 4, 3)), (5, (Q, 8, 256, 144)), (6, (F, 8, 3, 3)), (7, (F, 5, 256)), (8, (F, 1024))],
}


def tensors(args, device_of=lambda k: 0):
    return [Fake(*a, device=device_of(i)) if isinstance(a, tuple) else a for i, a in enumerate(args)]


@pytest.mark.parametrize("name", GOOD)
def test_binding_refuses_tensors_that_do_not_fit(calls, name):
    fn = getattr(calls, name)
    assert fn(*tensors(GOOD[name])) == 0
    for at, wrong in WRONG[name]:
        args = list(GOOD[name])
        args[at] = wrong
        with pytest.raises((ValueError, TypeError)):
            fn(*tensors(args))
    for at, a in enumerate(GOOD[name]):
        if isinstance(a, tuple):
            for device in (1, -1):
                with pytest.raises(ValueError, match="CUDA device"):
                    fn(*tensors(GOOD[name], lambda k: device if k == at else 0))


def test_binding_refuses_strides_that_the_calls_do_not_take(calls):
    x, xs, w, ws, y, stream = tensors(GOOD["fp8_gemm"])
    assert calls.fp8_gemm(Fake(Q, 5, 272, stride=(288, 1)), xs, w, ws, Fake(B, 5, 130, stride=(200, 1)), stream) == 0
    for bad in (Fake(Q, 5, 272, stride=(1, 5)), Fake(Q, 5, 272, stride=(544, 2))):
        with pytest.raises(ValueError, match="dense rows"):
            calls.fp8_gemm(bad, xs, w, ws, y, stream)
    with pytest.raises(ValueError, match="contiguous"):
        calls.fp8_gemm(x, xs, Fake(Q, 130, 272, stride=(288, 1)), ws, y, stream)
    with pytest.raises(ValueError, match="contiguous"):
        calls.fp8_gemm(x, xs, w, Fake(F, 2, 3, stride=(1, 2)), y, stream)


def test_binding_refuses_host_tensors():
    import mmvq_q2_gb300 as q
    x = torch.zeros(2, 256)
    with pytest.raises(ValueError, match="CUDA"):
        q.fp8_quantize(x)
    with pytest.raises(ValueError, match="block_rows"):
        q.fp8_quantize(x, block_rows=64)
    with pytest.raises(ValueError, match="CUDA"):
        q.swiglu_fp8_rows(x)
    code = x.to(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="CUDA"):
        q.fp8_gemm(code, x, code, x)
    with pytest.raises(ValueError, match="CUDA"):
        q.fp8_moe(x.bfloat16(), x, x, code, x, code, x)
