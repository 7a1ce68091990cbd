"""Rules of the kernels over 8-bit floating-point operands that no input can
show at run time, read from their sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mmvq_q2_gb300", "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def kernels(name):
    """The bodies of the kernels in a source, without comments."""
    text, out = source(name), {}
    for m in re.finditer(r"__global__ void __launch_bounds__\(.*?\)\s+(\w+)\(const", text, re.S):
        at = text.index("{", text.index(")\n{", m.end()))
        out[m.group(1)] = text[at:text.index("\n}\n", at)]
    return out


@pytest.mark.parametrize("name,count", [("fp8_ops.cu", 4), ("fp8_gemm.cu", 1), ("fp8_stream.cu", 1)])
def test_no_block_leaves_before_it_has_waited_for_the_launch_before(name, count):
    found = kernels(name)
    assert len(found) == count
    for kernel, body in found.items():
        assert "pdl_wait();" in body, kernel
        first = re.search(r"\breturn;", body)
        assert first is None or body.index("pdl_wait();") < first.start(), kernel


def test_what_reads_ahead_of_its_wait_starts_after_all_before_is_complete():
    """The second launch of fp8_moe reads ids and weights before it waits, so the first may let it start only once it has
    waited itself."""
    body = kernels("fp8_stream.cu")["fp8_stream_kernel"]
    assert body.index("if (MODE != DOWN)\n        pdl_wait();") < body.index("pdl_launch_dependents();")


def test_every_wait_on_a_barrier_has_a_limit():
    for name in ("fp8_gemm.cu", "fp8_stream.cu"):
        assert "mbar_try_wait(" not in source(name) and "mbar_wait_near(" in source(name)
    assert "2000000000ull" in source("fp8_common.cuh")


def test_registers_moved_between_warps_add_up():
    """setmaxnreg draws on what the block was launched with: 384 threads of at most 168."""
    text = source("fp8_gemm.cu")
    down, up = (int(re.search(rf"setmaxnreg\.{way}\.sync\.aligned\.u32 (\d+)", text).group(1)) for way in ("dec", "inc"))
    threads = int(re.search(r"kThreads = (\d+)", text).group(1))
    launched = 65536 // threads // 8 * 8
    assert 128 * down + (threads - 128) * up <= threads * launched


def test_no_second_block_with_tensor_memory_fits_beside_one():
    """Every launch of a kernel that takes all of tensor memory asks for all but 8 KB of shared memory: two blocks on one
    SM would wait for each other's tensor memory, and across two clusters for ever."""
    for name in ("fp8_gemm.cu", "fp8_stream.cu"):
        asked = re.findall(r"dynamicSmemBytes = ([^;]+);", source(name))
        assert asked
        for size in asked:
            assert size.startswith("alone_on_sm(") or size == "(size_t)di.smem_optin", (name, size)
    assert "most - 8192;" in source("fp8_common.cuh")
