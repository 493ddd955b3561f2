"""What one attention kernel may see of another's output, read off the source: with programmatic launch a kernel's CTAs
may be there before the kernels ahead are done, so that nothing those write may pass the non-coherent path, and
k_attn_dq, which works before its wait for the kernel ahead, needs an order of its own behind delta's kernel."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bwd_adapter_adamw_gb300", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(src, head):
    """The braces behind the first `head`."""
    at = src.index("{", src.index(")", src.index(head)))
    depth = 0
    for i in range(at, len(src)):
        depth += {"{": 1, "}": -1}.get(src[i], 0)
        if depth == 0:
            return src[at:i + 1]
    raise AssertionError(head)


@pytest.mark.parametrize("name", ["attn_common.cuh", "attention.cu", "attention_bwd.cu"])
def test_no_read_of_a_kernels_output_is_non_coherent(name):
    assert not re.search(r"__ldg\b|ld\.global\.nc", code(name))


def test_dq_acquires_what_dkv_released_behind_its_wait():
    src = code("attention_bwd.cu")
    dep = body(src, "void dkv_dep_sync")
    assert dep.index("griddepcontrol.wait") < dep.index("flag_set") < dep.index("griddepcontrol.launch_dependents")
    dkv = body(src, "k_attn_dkv(const")
    assert "griddepcontrol" not in dkv and not re.search(r"\bgrid_dep_sync", dkv) and dkv.count("dkv_dep_sync") == 2
    assert "*ready = 0" in body(src, "k_attn_delta(const").split("grid_dep_sync();")[1]
    dq = body(src, "k_attn_dq(const")
    order = [dq.index(s) for s in ("flag_wait", "__syncthreads", "fence.proxy.async", "Items items", "items.n = 0", "items.take",
                                   "griddepcontrol.wait")]
    assert order == sorted(order)
    common = code("attn_common.cuh")
    assert "st.release.gpu" in body(common, "void flag_set") and "ld.acquire.gpu" in body(common, "bool flag_wait")
