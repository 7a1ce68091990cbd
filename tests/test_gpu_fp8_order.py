"""fp8_moe right behind launches of this library that let what follows start
before they are complete: what they wrote counts, in every replay."""
import pytest
import torch

from test_gpu_fp8 import BF16, DEV, F32, gen, lib, moe_inputs, normal  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,E,topk,dim,inter", [(1, 64, 4, 512, 256), (6, 16, 3, 256, 384), (32, 64, 8, 640, 128), (64, 8, 4, 256, 128)])
def test_moe_behind_the_route_that_writes_its_ids(lib, m, E, topk, dim, inter):  # noqa: F811
    """moe_route_topk starts its dependents at once; its ids and weights change with each step, in the same buffers, and
    so does x, which norm_gate_residual writes."""
    args = moe_inputs(m, m, E, topk, dim, inter)
    experts, steps = args[3:], 8
    logits = [normal(gen(100 + i), m, E) for i in range(steps)]
    h = [normal(gen(200 + i), m, dim) for i in range(steps)]
    weight = torch.ones(dim, device=DEV)
    want = []
    for i in range(steps):
        ids, w = lib.moe_route_topk(logits[i], topk)
        torch.cuda.synchronize()
        want.append(lib.fp8_moe(norm(lib, h[i], weight), ids, w, *experts))
        torch.cuda.synchronize()
    assert all(not torch.equal(want[i], want[i + 1]) for i in range(steps - 1))
    ids, w = (torch.empty((m, topk), dtype=t, device=DEV) for t in (torch.int32, F32))
    x = torch.empty((m, dim), dtype=BF16, device=DEV)
    got = [torch.empty((m, dim), device=DEV) for _ in range(steps)]
    work = torch.empty(lib.fp8_moe_workspace_bytes(m, topk, dim, inter), dtype=torch.uint8, device=DEV)

    def all_steps():
        for i in range(steps):
            norm(lib, h[i], weight, x)
            lib.moe_route_topk(logits[i], topk, ids=ids, weights=w)
            lib.fp8_moe(x, ids, w, *experts, out=got[i], workspace=work)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        all_steps()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        with torch.cuda.graph(graph, stream=side):
            all_steps()
    for _ in range(20):
        for y in got:
            y.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def norm(lib, h, weight, out=None):  # noqa: F811
    return lib.norm_gate_residual(h, weight, 1e-6, out=out)[1]
