"""Rules of the decode-layer kernels that no input can show at run time: what
has to have happened before a block may leave.  Read from the sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mmvq_q2_gb300", "csrc")


def kernels(name):
    """The bodies of the kernels in a source, without comments."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    out = {}
    for m in re.finditer(r"__global__ void __launch_bounds__\(.*?\)\s+(\w+)\(", text, re.S):
        at = text.index("{", text.index(")\n{", m.end()))
        end = text.index("\n}\n", at)
        out[m.group(1)] = text[at:end]
    return out


@pytest.mark.parametrize("name", ["kv_page.cu", "kv_attn.cu", "layer_ops.cu"])
def test_no_block_leaves_before_it_has_waited_for_the_launch_before(name):
    """A grid that completes without griddepcontrol.wait lets its dependents run beside what it should have followed."""
    found = kernels(name)
    assert len(found) >= 2
    for kernel, body in found.items():
        assert "pdl_wait();" in body, kernel
        first = re.search(r"\breturn;", body)
        assert first is None or body.index("pdl_wait();") < first.start(), kernel


def test_attention_leaves_no_piece_header_unset():
    """The join takes heads[x] for an item of pieces unless it says -1: every block sets its own before it may leave."""
    body = kernels("kv_attn.cu")["kv_attn_kernel"]
    first = re.search(r"\breturn;", body)
    assert body.index("a.heads[blockIdx.x].first = -1;") < first.start()
