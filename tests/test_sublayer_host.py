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
