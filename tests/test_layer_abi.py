"""The decode-layer calls (page plan, rotary store, paged attention, fused
norms, expert routing) refuse bad arguments with a status before any launch,
and their binding refuses tensors that do not fit.  CPU only."""
import ctypes
import math

import pytest
import torch

P = ctypes.c_void_p
A = P(0x10000)      # never dereferenced: validation fails first
ODD = P(0x10001)
H4 = P(0x10004)     # 4-byte aligned only
NULL, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 6


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


def test_page_plan_refusals(L):
    # ctx, new, n_req, page, free, n_free, head, table, cols, ld, cu, seq, pos, req, slot, max_tokens,
    # head_out, err, stream
    good = (A, A, 4, 16, A, 10, None, A, 8, 8, A, A, A, A, A, 4, A, None, None)
    refused(L.kv_page_plan, good, [
        ({0: None}, NULL), ({1: None}, NULL), ({4: None}, NULL), ({7: None}, NULL), ({10: None}, NULL),
        ({11: None}, NULL), ({12: None}, NULL), ({13: None}, NULL), ({14: None}, NULL), ({16: None}, NULL),
        ({2: 0}, SHAPE), ({2: 16385}, SHAPE), ({3: 24}, SHAPE), ({3: 8}, SHAPE), ({3: 2048}, SHAPE), ({5: -1}, SHAPE),
        ({8: 0}, SHAPE), ({9: 7}, SHAPE), ({15: -1}, SHAPE), ({15: (1 << 30) + 1}, SHAPE),
        ({6: P(0x20000), 16: P(0x20000)}, SHAPE),  # free_head and free_head_out are two places
        ({0: ODD}, ALIGN), ({7: ODD}, ALIGN), ({14: ODD}, ALIGN), ({17: ODD}, ALIGN),
    ])


def test_rope_store_refusals(L):
    sec = (ctypes.c_int32 * 3)(16, 24, 24)
    # q, ld_q, k, ld_k, v, ld_v, type, T, Hq, Hkv, D, pos, n_axes, sections, inv_freq, rot, interleaved, slots,
    # q_out, ld_qo, k_cache, v_cache, n_pages, page, page_stride, err, stream
    good = (A, 512, A, 256, A, 256, 0, 3, 4, 2, 128, A, 3, sec, A, 128, 0, A, A, 512, A, A, 10, 16, 4096, None, None)
    refused(L.kv_rope_store, good, [
        ({0: None}, NULL), ({18: None}, NULL), ({2: None}, NULL), ({4: None}, NULL), ({11: None}, NULL),
        ({13: None}, NULL), ({14: None}, NULL), ({17: None}, NULL), ({20: None}, NULL), ({21: None}, NULL),
        ({6: 2}, SHAPE), ({7: -1}, SHAPE), ({8: 0}, SHAPE), ({9: 0}, SHAPE), ({10: 513}, SHAPE), ({10: 0}, SHAPE),
        ({12: 0}, SHAPE), ({12: 4}, SHAPE), ({12: 1}, SHAPE), ({15: 126}, SHAPE),
        ({15: 127}, SHAPE), ({15: 130}, SHAPE), ({16: 2}, SHAPE), ({1: 511}, SHAPE), ({3: 255}, SHAPE),
        ({5: 255}, SHAPE), ({19: 511}, SHAPE), ({22: 0}, SHAPE), ({22: 1 << 28}, SHAPE), ({23: 48}, SHAPE),
        ({24: 4095}, SHAPE), ({24: 4100}, SHAPE),
        ({0: P(0x10002)}, ALIGN), ({20: ODD}, ALIGN), ({17: ODD}, ALIGN),
    ])
    bad = (ctypes.c_int32 * 3)(-1, 41, 24)
    refused(L.kv_rope_store, good, [({13: bad}, SHAPE)])


def test_attention_refusals(L):
    need = L.kv_attention_workspace_bytes(4, 8, 2, 128)
    assert need > 0
    for bad in ((-1, 8, 2, 128), (4, 8, 3, 128), (4, 8, 0, 128), (4, 8, 2, 100), (4, 8, 2, 144), (4, 8, 2, 0),
                (4, 258, 2, 128), ((1 << 24) + 1, 8, 2, 128)):
        assert L.kv_attention_workspace_bytes(*bad) == 0, bad
    # q, ld_q, T, Hq, Hkv, D, k, v, n_pages, page, page_stride, table, cols, ld, cu, seq, n_req, scale, window,
    # out, ld_o, lse, workspace, bytes, stream
    good = (A, 1024, 4, 8, 2, 128, A, A, 10, 16, 4096, A, 8, 8, A, A, 2, 0.1, 0, A, 1024, None, A, need, None)
    refused(L.kv_attention_bf16, good, [
        ({0: None}, NULL), ({6: None}, NULL), ({7: None}, NULL), ({11: None}, NULL), ({14: None}, NULL),
        ({15: None}, NULL), ({19: None}, NULL),
        ({2: -1}, SHAPE), ({3: 7}, SHAPE), ({4: 0}, SHAPE), ({5: 120}, SHAPE), ({5: 144}, SHAPE), ({1: 1016}, SHAPE),
        ({1: 1028}, SHAPE), ({20: 1023}, SHAPE), ({8: 0}, SHAPE), ({9: 17}, SHAPE), ({10: 4088}, SHAPE),
        ({12: 0}, SHAPE), ({13: 7}, SHAPE), ({16: -1}, SHAPE), ({16: 16385}, SHAPE), ({17: 0.0}, SHAPE), ({17: -1.0}, SHAPE),
        ({17: math.nan}, SHAPE), ({17: math.inf}, SHAPE), ({18: -1}, SHAPE),
        ({22: None}, WORKSPACE), ({23: need - 1}, WORKSPACE),
        ({0: P(0x10008)}, ALIGN), ({6: P(0x10008)}, ALIGN), ({7: H4}, ALIGN), ({11: ODD}, ALIGN), ({19: ODD}, ALIGN),
        ({21: P(0x10002)}, ALIGN), ({22: P(0x10010)}, ALIGN),
    ])


def test_norm_refusals(L):
    # y, y_type, ld_y, post_w, gate, ld_gate, residual, s_type, ld_res, alpha, pre_w, eps, T, dim, residual_out, ld_ro,
    # out, ld_out, out_q8, stream
    good = (A, 0, 64, A, A, 0, A, 1, 64, 1.0, A, 1e-6, 3, 64, A, 64, A, 64, A, None)
    refused(L.norm_gate_residual, good, [
        ({6: None}, NULL), ({10: None}, NULL), ({0: None}, NULL), ({14: None, 16: None, 18: None}, NULL),
        ({1: 2}, SHAPE), ({7: -1}, SHAPE), ({12: -1}, SHAPE), ({13: 0}, SHAPE), ({13: 32769}, SHAPE), ({2: 63}, SHAPE),
        ({5: 63}, SHAPE), ({8: 63}, SHAPE), ({15: 63}, SHAPE), ({17: 63}, SHAPE), ({11: -1.0}, SHAPE),
        ({11: math.nan}, SHAPE), ({9: math.inf}, SHAPE), ({9: math.nan}, SHAPE), ({13: 48}, SHAPE),
        ({0: P(0x10002)}, ALIGN), ({6: ODD}, ALIGN), ({10: P(0x10002)}, ALIGN), ({18: P(0x10002)}, ALIGN),
    ])


def test_route_refusals(L):
    # logits, type, m, E, ld, bias, score, n_group, topk_group, topk, renorm, scale, ids, weights, ptrs, ptrs_out, stream
    good = (A, 0, 3, 64, 64, None, 0, 8, 2, 8, 1, 1.0, A, A, A, A, None)
    refused(L.moe_route_topk, good, [
        ({0: None}, NULL), ({12: None}, NULL), ({13: None}, NULL), ({14: None}, NULL), ({15: None}, NULL),
        ({1: 2}, SHAPE), ({2: -1}, SHAPE), ({3: 0}, SHAPE), ({3: 1025, 4: 1025}, SHAPE), ({4: 63}, SHAPE),
        ({6: 2}, SHAPE), ({7: 0}, SHAPE), ({7: 7}, SHAPE), ({7: 64}, SHAPE), ({8: 0}, SHAPE), ({8: 9}, SHAPE),
        ({9: 0}, SHAPE), ({9: 17}, SHAPE), ({8: 8, 9: 33}, SHAPE), ({10: 2}, SHAPE), ({11: math.nan}, SHAPE),
        ({0: P(0x10002)}, ALIGN), ({5: ODD}, ALIGN), ({14: H4}, ALIGN),
    ])


def test_binding_refuses_host_tensors_and_wrong_types():
    import mmvq_q2_gb300 as q
    x = torch.zeros(2, 4, 16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        q.moe_route_topk(torch.zeros(2, 8), 2)
    with pytest.raises(ValueError, match="CUDA"):
        q.norm_gate_residual(torch.zeros(2, 8), torch.zeros(8), 1e-6)
    with pytest.raises(ValueError, match="CUDA"):
        q.kv_page_plan(i, i, 16, i, torch.zeros(2, 4, dtype=torch.int32), 2)
    with pytest.raises(ValueError, match="CUDA"):
        q.kv_rope_store(x, x, x, i, torch.zeros(8), i, torch.zeros(1, 4, 16, 16), torch.zeros(1, 4, 16, 16))
    with pytest.raises(ValueError, match="CUDA"):
        q.kv_attention_bf16(x.bfloat16(), torch.zeros(1, 4, 16, 16), torch.zeros(1, 4, 16, 16), i, i, i)
