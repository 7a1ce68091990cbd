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
