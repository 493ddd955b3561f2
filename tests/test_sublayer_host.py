"""Host-side behaviour of the operators around the adapted linear and of the step that runs them:
refusals, memory that runs out, what the step hands to the library. No GPU."""
import os
import subprocess
import sys

import pytest

FAKE = 1 << 20   # an aligned non-null address; never dereferenced (validation fails first)
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    from bwd_adapter_adamw_gb300 import build
    build.build()
    from bwd_adapter_adamw_gb300 import binding
    return binding


@pytest.mark.parametrize("offset", [(1 << 63) - 4, (1 << 63) - 512, (1 << 62), 2048 + 4, 2048])
def test_update_refuses_matrices_whose_end_overflows(L, offset):
    groups = L.make_groups([dict(offset=0, n_a=1024, n_b=1024, grad_scale=1.0, lr=0.1)])
    mats = L.make_mats([dict(offset=offset, rows=8, cols=64, kind=L.LORA_KIND_A)])
    assert L.lora_muon_step(FAKE, FAKE, FAKE, groups, mats, L.make_muon_hp(), FAKE, FAKE, False, FAKE, 1 << 30,
                            stream=0, check=False) == L.LORA_ERR_INVALID


def test_memory_that_runs_out_is_a_status(L):
    """Two million matrices with 24 MB of address space left: the update's host tables do not fit."""
    code = """
import ctypes as C, resource, sys
import numpy as np
sys.path.insert(0, %r)
from bwd_adapter_adamw_gb300 import binding as L
n = 2000000
a = np.zeros(n, dtype=[("offset", "i8"), ("rows", "i8"), ("cols", "i8"), ("group", "i4"), ("kind", "i4")])
assert a.itemsize == C.sizeof(L.lora_mat)
a["offset"], a["rows"], a["cols"] = 16 * np.arange(n), 4, 4
mats = (L.lora_mat * n).from_buffer(a)
groups = L.make_groups([dict(offset=0, n_a=16 * n, grad_scale=1.0, lr=0.1)])
back = (L.lora_mat * n).from_buffer(a[::-1].copy())
size = [int(l.split()[1]) for l in open("/proc/self/status") if l.startswith("VmSize")][0] << 10
resource.setrlimit(resource.RLIMIT_AS, (size + (24 << 20), resource.getrlimit(resource.RLIMIT_AS)[1]))
F = 1 << 20
assert L.lora_muon_workspace_size(mats) == 0
assert L.lora_muon_workspace_size(back) == 0
for m in (mats, back):
    st = L.lora_muon_step(F, F, F, groups, m, L.make_muon_hp(), F, F, False, F, 1 << 30, stream=0, check=False)
    assert st == L.LORA_ERR_UNSUPPORTED, st
print("ok")
""" % ROOT
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stderr[-500:])
