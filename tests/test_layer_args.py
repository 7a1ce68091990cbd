"""Arguments that the decode-layer calls and their binding have to refuse
before any launch.  CPU only: no address here is dereferenced."""
import ctypes

import pytest

P = ctypes.c_void_p
SHAPE = 2


@pytest.fixture(scope="module")
def L():
    from mmvq_q2_gb300 import build
    build.build()
    import mmvq_q2_gb300 as q
    return q.lib()


def test_page_plan_refuses_outputs_over_its_inputs(L):
    # ctx, new, n_req, page, free, n_free, head, table, cols, ld, cu, seq, pos, req, slot, max_tokens, head_out, err
    count = {0: 4, 1: 4, 4: 10, 6: 1, 10: 5, 11: 4, 12: 6, 13: 6, 14: 6, 16: 1, 17: 1}
    at = {i: 0x10000 + 0x100 * i for i in count}
    for i in (0, 1, 4, 6):
        for o in (10, 11, 12, 13, 14, 16, 17):
            # in the same place, the output's last entry on the first, its first on the last
            for where in (at[i], at[i] - 4 * (count[o] - 1), at[i] + 4 * (count[i] - 1)):
                a = dict(at)
                a[o] = where
                args = [P(a[0]), P(a[1]), 4, 16, P(a[4]), 10, P(a[6]), P(0x90000), 8, 8, P(a[10]), P(a[11]), P(a[12]),
                        P(a[13]), P(a[14]), 6, P(a[16]), P(a[17]), None]
                assert L.kv_page_plan(*args) == SHAPE, (i, o, where - at[i])


class Fake:
    """What the binding reads off a tensor: no memory, any device."""

    def __init__(self, dtype, *shape, device=0):
        import torch
        self.dtype, self.shape, self.device_index = getattr(torch, dtype), shape, device
        self.is_cuda = device >= 0

    def stride(self):
        out, n = [], 1
        for s in reversed(self.shape):
            out.insert(0, n)
            n *= s
        return tuple(out)

    def data_ptr(self):
        return 0x10000

    def get_device(self):
        return self.device_index


@pytest.fixture
def calls(L):
    """The binding's native half over functions that do nothing; the current device is 0."""
    import torch

    import mmvq_q2_gb300 as q
    m = q._calls()
    nothing = ctypes.CFUNCTYPE(ctypes.c_int)(lambda: 0)
    types = torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8
    try:
        m.setup(types, (ctypes.cast(nothing, P).value,) * 6, lambda: 0)
        yield m
    finally:
        q._native = None
        q._calls()


def device_cases():
    f, b, i = "float32", "bfloat16", "int32"
    cache = [(b, 4, 2, 16, 64)] * 2
    return {
        "kv_page_plan": [(i, 3), (i, 3), 16, (i, 9), (i, 1), (i, 3, 4), 5, ((i, 4), (i, 3), (i, 5), (i, 5), (i, 5), (i, 1)),
                         (i, 1), 0],
        "kv_rope_store": [(f, 5, 4, 64), (f, 5, 2, 64), (f, 5, 2, 64), (i, 5), (f, 32), (i, 5), *cache, (32,), False,
                          (b, 5, 4, 64), (i, 1), 0],
        "kv_attention_bf16": [(b, 5, 4, 64), *cache, (i, 3, 4), (i, 4), (i, 3), None, 0, (b, 5, 4, 64), (f, 5, 4),
                              ("uint8", 64), 0],
        "norm_gate_residual": [(f, 5, 64), (f, 64), 1e-6, (f, 5, 64), (f, 64), (f, 64), 1.0, (f, 5, 64), (b, 5, 64),
                               ("uint8", 5, 72), 0],
        "moe_route_topk": [(f, 5, 16), 2, (f, 16), 0, 1, 1, True, 1.0, (i, 5, 2), (f, 5, 2), ("int64", 3, 16),
                           ("int64", 5, 6), 0],
    }


def is_spec(a):
    return isinstance(a, tuple) and isinstance(a[0], str)


def faked(args, device_of):
    """The arguments with tensors in the place of their shapes, the n-th on device_of(n); and how many there are."""
    count = 0

    def one(a):
        nonlocal count
        if is_spec(a):
            count += 1
            return Fake(*a, device=device_of(count - 1))
        return tuple(one(x) for x in a) if isinstance(a, tuple) and a and is_spec(a[0]) else a

    return [one(a) for a in args], count


@pytest.mark.parametrize("name", device_cases())
def test_binding_refuses_tensors_of_another_device(calls, name):
    fn, args = getattr(calls, name), device_cases()[name]
    good, n = faked(args, lambda k: 0)
    assert fn(*good) == 0 and n >= 6
    for wrong in range(n):
        with pytest.raises(ValueError, match="current CUDA device"):
            fn(*faked(args, lambda k: 1 if k == wrong else 0)[0])
        with pytest.raises(ValueError, match="must be on a CUDA device"):
            fn(*faked(args, lambda k: -1 if k == wrong else 0)[0])
    # all of one device, but not of the current one, where the kernels would run
    with pytest.raises(ValueError, match="current CUDA device"):
        fn(*faked(args, lambda k: 1)[0])
